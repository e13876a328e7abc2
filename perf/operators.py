"""The adapter, rotary and 8-bit-cache operators as work to be measured: cases, inputs, and each operator twice over.

`own` false: the operator in plain torch operations in 32 bits (64 where 32 lose what matters), rounded once at the
end.  `own` true: the calls a user makes of liblowbit's entry points.  `exact` is the definition in 64 bits, written
apart from the plain form.  The operators (include/lowbit.h has the definitions):

  lora    y[m] = base[m] + s_i B_i (A_i x[m]) with i = ids[m]; rows whose id names no adapter keep base
  rope    rotary positions on query and key heads: pairs (j, j + rot/2) or (2j, 2j+1) of the first rot entries of a head
  write   new keys and values into pages of int8 codes with one scale per page and head, and the touched pages read back
  attend  attention of each sequence's newest rows over its pages, causal, grouped heads
"""
import math
import random

import torch

own = False

DEV = "cuda"
WORKSPACE = 64 << 20


# -- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one request decoding through one 4096-wide projection: the smallest call, latency alone counts
        {"name": "lora one token", "op": "lora", "rows": 1, "adapters": 8, "rank": 16, "k": 4096, "n": 4096, "targets": 1},
        # a decode batch, each request with an adapter of its own, over the query, key and value projections at once
        {"name": "lora decode q,k,v", "op": "lora", "rows": 16, "adapters": 32, "rank": 16, "k": 5120, "n": 5120, "targets": 3},
        # a larger decode batch on the wide feed-forward projections (gate and up), adapters of several ranks
        {"name": "lora decode wide", "op": "lora", "rows": 61, "adapters": 48, "rank": 64, "k": 5120, "n": 17408, "targets": 2},
        # prompts of several requests through a feed-forward projection: bound by reading base and writing y
        {"name": "lora prompts", "op": "lora", "rows": 4096, "adapters": 8, "rank": 32, "k": 4096, "n": 11008, "targets": 1},
        # a decode step's queries and keys as the projections leave them (32 bits), positions far into a scaled context
        {"name": "rope decode far", "op": "rope", "rows": 64, "q_heads": 40, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "from32": True, "far": 1 << 20, "scaled": True},
        # prompts, half of each head rotated, interleaved pairs, 16-bit input
        {"name": "rope prompts", "op": "rope", "rows": 8191, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 64,
         "interleaved": True, "from32": False, "far": 1 << 15, "scaled": False},
        # a decode step writes one token of each sequence
        {"name": "write decode", "op": "write", "seqs": 64, "rows_max": 1, "kv_max": 8192, "kv_heads": 8, "dim": 128, "page": 64},
        # prompts of several requests written at once
        {"name": "write prompts", "op": "write", "seqs": 7, "rows_max": 2500, "kv_max": 4096, "kv_heads": 8, "dim": 128, "page": 32},
        # one request, a short context: latency
        {"name": "attend one short", "op": "attend", "seqs": 1, "rows_max": 1, "kv_max": 777, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64},
        # a decode batch of ragged contexts (an idle slot among them)
        {"name": "attend decode batch", "op": "attend", "seqs": 64, "rows_max": 1, "kv_max": 8192, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 64},
        # one request, a long context, several proposed tokens checked at once
        {"name": "attend long check", "op": "attend", "seqs": 1, "rows_max": 4, "kv_max": 131071, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 128},
        # prompt chunks over what is cached already: bound by arithmetic
        {"name": "attend prompts", "op": "attend", "seqs": 3, "rows_max": 1900, "kv_max": 8192, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "rope", "write", "attend", "attend"])
    if op == "lora":
        rows = _log(rng, 1, 4096)
        return {"op": op, "rows": rows, "adapters": rng.randint(1, 8 if rows > 256 else 48), "rank": rng.choice([8, 16, 24, 32, 64] if rows <= 256 else [8, 16, 32]),
                "k": 64 * rng.randint(8, 80 if rows <= 256 else 64), "n": 8 * _log(rng, 64, 2176 if rows <= 256 else 1376), "targets": rng.randint(1, 3) if rows <= 256 else 1}
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        return {"op": op, "rows": _log(rng, 1, 8192), "q_heads": rng.randint(1, 8) * 2, "kv_heads": rng.choice([1, 2, 4, 8]), "dim": dim, "rot": rng.choice([dim, dim // 2, dim // 4]),
                "interleaved": rng.random() < 0.5, "from32": rng.random() < 0.5, "far": _log(rng, 1 << 10, 1 << 20), "scaled": rng.random() < 0.5}
    kv_heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([32, 64, 128])
    if op == "write":
        many = rng.random() < 0.5
        return {"op": op, "seqs": _log(rng, 1, 8 if many else 128), "rows_max": _log(rng, 2, 2048) if many else 1, "kv_max": _log(rng, 2100, 8192),
                "kv_heads": kv_heads, "dim": dim, "page": page}
    kind = rng.choice(["decode", "long", "check", "prompts"])
    group = rng.choice([1, 2, 4, 5, 8])
    case = {"op": op, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page}
    if kind == "decode":
        return case | {"seqs": _log(rng, 2, 64), "rows_max": 1, "kv_max": _log(rng, 17, 8192)}
    if kind == "long":
        return case | {"seqs": rng.randint(1, 2), "rows_max": 1, "kv_max": _log(rng, 8192, 65536)}
    if kind == "check":
        return case | {"seqs": _log(rng, 1, 16), "rows_max": rng.randint(2, 8), "kv_max": _log(rng, 64, 16384)}
    return case | {"seqs": rng.randint(1, 3), "rows_max": _log(rng, 65, 1024), "kv_max": _log(rng, 1024, 8192)}


def _lengths(case):
    """(rows, cached tokens with the new rows) of every sequence, from the case alone."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["rows_max"], case["kv_max"]))
    B, most, far = case["seqs"], case["rows_max"], case["kv_max"]
    rows = [most if b == 0 else rng.randint(max(1, most // 4), most) for b in range(B)]
    kv = [far if b == 0 else max(rows[b], _log(rng, max(1, far // 16), far)) for b in range(B)]
    if B >= 8 and most == 1:
        kv[B // 2], rows[B // 2] = (0, 1) if case["op"] == "attend" else (1, 1)  # an idle slot; a sequence's first token
    return rows, kv


def _touched(case):
    """Tokens of the pages that a write touches, for every sequence: from the start of the first touched page on."""
    rows, kv = _lengths(case)
    return [n + (t - n) % case["page"] for n, t in zip(rows, kv)]


def work(case):
    op = case["op"]
    if op == "lora":
        M, R, r, K, N = case["rows"], case["targets"], case["rank"], case["k"], case["n"]
        ids, ranks = _ids(case), _ranks(case)
        used = sorted({i for i in ids if i >= 0})
        weights = sum(ranks[i] * (K + N) * 2 for i in used)
        flops = sum(2 * ranks[i] * (K + N) for i in ids if i >= 0)
        return {"bytes": R * (weights + 8 * M * N) + 2 * M * K, "flops": R * flops}
    if op == "rope":
        values = case["rows"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": values * ((4 if case["from32"] else 2) + 2) + 4 * case["rows"], "flops": 3 * values}
    rows, kv = _lengths(case)
    H, D = case["kv_heads"], case["dim"]
    if op == "write":
        new, back = sum(rows) * H * D, sum(_touched(case)) * H * D
        return {"bytes": new * (2 + 4) + 2 * new + 2 * back * (1 + 4), "flops": 6 * new + 2 * back}
    Q = case["q_heads"]
    seen = sum(n * t - n * (n - 1) // 2 for n, t in zip(rows, kv) if t)
    pages = sum(-(-t // case["page"]) for t in kv)
    return {"bytes": 2 * sum(kv) * H * D + 8 * pages * H + 4 * sum(rows) * Q * D, "flops": 4 * seen * Q * D}


# -- inputs -----------------------------------------------------------------------------------------------------------

def _ids(case):
    """The adapter of every row: requests of a decode batch in any order, prompts in runs; a few rows without one."""
    rng = random.Random("%d %d" % (case["rows"], case["adapters"]))
    M, L = case["rows"], case["adapters"]
    if M <= 256:
        ids = [rng.randrange(L) for _ in range(M)]
        return [-1 if M > 8 and m % 11 == 5 else i for m, i in enumerate(ids)]
    ids = []
    while len(ids) < M:
        ids += [rng.randrange(-1, L)] * rng.randint(M // 16, M // 6)
    return ids[:M]


def _ranks(case):
    r = case["rank"]
    return [r if i % 3 else max(1, r // (1 + i % 2) - i % 5) for i in range(case["adapters"])]


def _frequencies(case):
    """Angles per position (64 bits) of the rot/2 pairs; where scaled, slow ones 8 times slower, with a ramp between."""
    half = case["rot"] // 2
    f = [10000.0 ** (-j / half) for j in range(half)]
    if case["scaled"]:
        turns = [8192 * w / (2 * math.pi) for w in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / (32.0 - 1.0))) for t in turns]
        f = [w / 8.0 * (1 - c) + w * c for w, c in zip(f, keep)]
    return f, (0.1 * math.log(8.0) + 1.0) if case["scaled"] else 1.0


def _signed(u):
    return u - (1 << 64) if u >= 1 << 63 else u


def _quantised(g, pages, heads, page, dim):
    x = torch.randn((pages, heads, page, dim), generator=g, device=DEV)
    x.mul_(torch.rand((pages, heads, 1, 1), generator=g, device=DEV).mul_(1.5).add_(0.5))
    top = x.abs().amax((2, 3))
    s = top / 127.0
    return (x / s[:, :, None, None]).round_().clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": case}
    if op == "lora":
        M, R, L, r, K, N = (case[k] for k in ("rows", "targets", "adapters", "rank", "k", "n"))
        st["x"] = torch.randn((M, K), generator=g, device=DEV).bfloat16()
        st["a"] = [(torch.randn((L, r, K), generator=g, device=DEV) / math.sqrt(K)).bfloat16() for _ in range(R)]
        st["b"] = [(torch.randn((L, N, r), generator=g, device=DEV) / math.sqrt(r)).bfloat16() for _ in range(R)]
        st["base"] = [torch.randn((M, N), generator=g, device=DEV) for _ in range(R)]
        st["y"] = [torch.empty((M, N), device=DEV) for _ in range(R)]
        st["ids"] = torch.tensor(_ids(case), dtype=torch.int32, device=DEV)
        st["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device=DEV)
        st["scales"] = torch.rand(L, generator=g, device=DEV) + 0.5
        st["ws"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV)
        return st
    if op == "rope":
        M, D = case["rows"], case["dim"]
        into = torch.float32 if case["from32"] else torch.bfloat16
        st["q"] = torch.randn((M, case["q_heads"], D), generator=g, device=DEV).to(into)
        st["k"] = torch.randn((M, case["kv_heads"], D), generator=g, device=DEV).to(into)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"], dtype=torch.bfloat16), torch.empty_like(st["k"], dtype=torch.bfloat16)
        st["positions"] = torch.randint(0, case["far"], (M,), generator=g, device=DEV, dtype=torch.int32)
        f, st["magnitude"] = _frequencies(case)
        st["frequencies"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        # the same in whole 2^-64 parts of a turn per position
        st["phases"] = torch.tensor([_signed(int(round(w / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1)) for w in f], dtype=torch.int64, device=DEV)
        return st
    rows, kv = _lengths(case)
    B, H, D, P = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    need = [-(-t // P) for t in kv]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)  # what no sequence reaches is never looked at
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    st["k_codes"], st["k_scales"] = _quantised(g, pages, H, P, D)
    st["v_codes"], st["v_scales"] = _quantised(g, pages, H, P, D)
    st["table"] = table.to(DEV)
    st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    st["row_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    T = starts[-1]
    if op == "write":
        back = [0]
        for n in _touched(case):
            back.append(back[-1] + n)
        st["back_start"] = torch.tensor(back, dtype=torch.int32, device=DEV)
        st["k"] = (torch.randn((T, H, D), generator=g, device=DEV) * (torch.rand((T, 1, 1), generator=g, device=DEV) + 0.5)).bfloat16()
        st["v"] = torch.randn((T, H, D), generator=g, device=DEV)
        st["k_back"], st["v_back"] = torch.empty((back[-1], H, D), device=DEV), torch.empty((back[-1], H, D), device=DEV)
    else:
        st["q"] = torch.randn((T, case["q_heads"], D), generator=g, device=DEV).bfloat16()
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
        st["ws"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV)
    return st


# -- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _calls(state)
    return {"lora": _plain_lora, "rope": _plain_rope, "write": _plain_write, "attend": _plain_attend}[state["op"]](state)


def _calls(s):
    from decode_packed_bit_b200 import lowbit as lb
    op, c = s["op"], s["case"]
    if op == "lora":
        lb.lowbit_lora_add_group(s["x"], s["ids"], s["a"], s["b"], s["base"], s["y"], ranks=s["ranks"], scales=s["scales"], workspace=s["ws"])
        return s["y"]
    if op == "rope":
        lb.lowbit_rope(s["q"], s["q_out"], s["k"], s["k_out"], s["positions"], s["phases"], interleaved=c["interleaved"], magnitude=s["magnitude"])
        return s["q_out"], s["k_out"]
    if "cache" not in s:  # the handle that a program keeps beside its buffers
        s["cache"] = lb.KV8Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    cache = s["cache"]
    one = c["rows_max"] == 1
    if op == "write":
        lb.lowbit_kv8_append(cache, s["table"], s["kv_len"], s["k"], s["v"], row_start=None if one else s["row_start"])
        lb.lowbit_kv8_read(cache, s["table"], s["kv_len"], s["k_back"], s["v_back"], row_start=s["back_start"])
        return s["k_back"], s["v_back"], s["k_scales"], s["v_scales"]
    lb.lowbit_kv8_attention(cache, s["table"], s["kv_len"], s["q"], s["out"], s["scale"], row_start=None if one else s["row_start"], workspace=s["ws"])
    return s["out"]


def _plain_lora(s):
    ids, L = s["ids"].long(), s["a"][0].shape[0]
    r = s["a"][0].shape[1]
    x = s["x"].float()
    wanted = (ids[:, None] == torch.arange(L, device=DEV))[:, :, None] & (torch.arange(r, device=DEV) < s["ranks"][:, None])[None]
    factor = torch.where(wanted, s["scales"][None, :, None], 0.0)  # [M][L][r]
    return [base + ((x @ a.float().reshape(L * r, -1).T).reshape(-1, L, r) * factor).reshape(-1, L * r) @ b.float().transpose(1, 2).reshape(L * r, -1)
            for a, b, base in zip(s["a"], s["b"], s["base"])]


def _plain_rope(s):
    angle = torch.remainder(s["positions"].double()[:, None] * s["frequencies"], 2 * math.pi)
    cos, sin = (angle.cos() * s["magnitude"]).float()[:, None, :], (angle.sin() * s["magnitude"]).float()[:, None, :]
    rot = 2 * angle.shape[1]

    def turn(x):
        x = x.float()
        head, tail = x[..., :rot], x[..., rot:]
        if s["case"]["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = head[..., : rot // 2], head[..., rot // 2:]
            head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((head, tail), -1).bfloat16()

    return turn(s["q"]), turn(s["k"])


def _places(start, kv_len, table, T, P):
    """Page, slot and position of every row, and its sequence."""
    row = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:].long(), row, right=True)
    position = kv_len.long()[b] - start.long()[b + 1] + row
    return table.long()[b, position // P], position % P, position, b


def _plain_write(s):
    P, T = s["case"]["page"], s["k"].shape[0]
    page, slot, position, b = _places(s["row_start"], s["kv_len"], s["table"], T, P)
    first = (s["kv_len"] - (s["row_start"][1:] - s["row_start"][:-1])).long()[b]  # the sequence's first new position
    continued = (position // P) * P < first                                     # older tokens lie in this page
    back_page, back_slot, back_position, back_b = _places(s["back_start"], s["kv_len"], s["table"], s["k_back"].shape[0], P)
    old_first = (s["kv_len"] - (s["row_start"][1:] - s["row_start"][:-1])).long()[back_b]
    is_old = (back_position < old_first)[:, None, None]
    back_row = (s["row_start"][1:].long()[back_b] - (s["kv_len"].long()[back_b] - back_position)).clamp_min(0)

    def write(x, codes, scales):
        x = x.float()
        seven = torch.full((), 127.0, device=DEV)  # a tensor: a division, not a product with 1/127
        top = x.abs().amax(-1) / seven
        kept = torch.zeros_like(scales).index_reduce_(0, page, torch.where(continued[:, None], scales[page], 0.0), "amax")
        new = kept.index_reduce(0, page, top, "amax")
        grown = new[page]
        fresh = torch.where(grown[..., None] > 0, torch.round(x.double() / grown.double()[..., None]), 0.0).clamp(-127, 127)
        was, now = scales.double()[back_page][..., None], new.double()[back_page][..., None]
        old = torch.where(now > 0, torch.round(codes[back_page, :, back_slot].double() * was / now), 0.0)
        values = torch.where(is_old, old, fresh[back_row]).float() * new[back_page][..., None]
        touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=DEV).index_fill_(0, page, True)
        return values, torch.where(touched[:, None], new, scales)

    k, ks = write(s["k"], s["k_codes"], s["k_scales"])
    v, vs = write(s["v"], s["v_codes"], s["v_scales"])
    return k, v, ks, vs


def _plain_attend(s):
    c = s["case"]
    P, H, D, Q, B = c["page"], c["kv_heads"], c["dim"], c["q_heads"], c["seqs"]
    most, longest = c["rows_max"], s["table"].shape[1] * P
    T = s["q"].shape[0]
    start, kv_len = s["row_start"].long(), s["kv_len"].long()
    row = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:], row, right=True)
    at = row - start[b]
    q = torch.zeros((B, most, H, Q // H, D), device=DEV)
    q[b, at] = s["q"].float().reshape(T, H, Q // H, D)
    pages = s["table"].long().clamp_min(0)

    def whole(codes, scales):  # [B][H][longest][D]
        return (codes[pages].float() * scales[pages][..., None, None]).transpose(1, 2).reshape(B, H, longest, D)

    scores = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, H, -1, D), whole(s["k_codes"], s["k_scales"]).transpose(2, 3))
    scores = scores.mul_(s["scale"]).reshape(B, H, Q // H, most, longest)
    last = kv_len[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(most, device=DEV)  # [B][most]
    hidden = torch.arange(longest, device=DEV)[None, None] > last[..., None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(B, H, -1, longest), whole(s["v_codes"], s["v_scales"])).reshape(B, H, Q // H, most, D)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(B, most, Q, D)[b, at].bfloat16()


# -- the definition in 64 bits ----------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lora":
        ids, ranks = _ids(case), _ranks(case)
        outs = []
        for a, b, base in zip(s["a"], s["b"], s["base"]):
            y = base.double()
            for i in sorted({i for i in ids if i >= 0}):
                rows = torch.tensor([m for m, j in enumerate(ids) if j == i], device=DEV)
                t = s["x"][rows].double() @ a[i, : ranks[i]].double().T
                y[rows] += s["scales"][i].double() * (t @ b[i, :, : ranks[i]].double().T)
            outs.append(y)
        return outs
    if op == "rope":
        f, magnitude = _frequencies(case)
        theta = torch.outer(s["positions"].double(), torch.tensor(f, dtype=torch.float64, device=DEV))
        turned = torch.polar(torch.full_like(theta, magnitude), torch.remainder(theta, 2 * math.pi))[:, None, :]
        half = len(f)
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double()
            if case["interleaved"]:
                z = torch.complex(y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()) * turned
                y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :half].clone(), y[..., half:2 * half].clone()) * turned
                y[..., :half], y[..., half:2 * half] = z.real, z.imag
            outs.append(y)
        return outs
    rows, kv = _lengths(case)
    P, table = case["page"], s["table"].tolist()
    if op == "write":
        outs, scales_out = [], []
        for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
            scales = scales.double()
            parts, r0 = [], 0
            for b, (n, t) in enumerate(zip(rows, kv)):
                p0 = t - n
                for j in range(p0 // P, (t - 1) // P + 1):
                    lo, hi, page = max(p0, j * P), min(t, (j + 1) * P), table[b][j]
                    fresh = x[r0 + lo - p0:r0 + hi - p0].double()
                    old = codes[page, :, : lo - j * P].double().transpose(0, 1)
                    was = scales[page].clone()
                    # the scale is stored in 32 bits: this rounding belongs to the definition
                    now = (fresh.abs().amax((0, 2)) / 127.0).float().double()
                    now = torch.maximum(now, was) if lo > j * P else now
                    scales[page] = now
                    safe = torch.where(now > 0, now, 1.0)[None, :, None]
                    held = torch.cat((torch.round(old * was[None, :, None] / safe), torch.round(fresh / safe).clamp(-127, 127)))
                    parts.append(held * now[None, :, None])
                r0 += n
            outs.append(torch.cat(parts))
            scales_out.append(scales)
        return outs + scales_out
    Q, H, D = case["q_heads"], case["kv_heads"], case["dim"]
    out, r0 = [], 0
    for b, (n, t) in enumerate(zip(rows, kv)):
        if t == 0:
            out.append(torch.zeros((n, Q, D), dtype=torch.float64, device=DEV))
            r0 += n
            continue
        pages = torch.tensor(table[b][: -(-t // P)], device=DEV)
        heads = []
        hidden = torch.ones((n, t), dtype=torch.bool, device=DEV).triu(t - n + 1)
        for h in range(H):
            k = (s["k_codes"][pages, h].double() * s["k_scales"][pages, h].double()[:, None, None]).reshape(-1, D)[:t]
            v = (s["v_codes"][pages, h].double() * s["v_scales"][pages, h].double()[:, None, None]).reshape(-1, D)[:t]
            for j in range(h * (Q // H), (h + 1) * (Q // H)):
                z = (s["q"][r0:r0 + n, j].double() @ k.T) * s["scale"]
                heads.append(torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v)
        out.append(torch.stack(heads, 1))
        r0 += n
    return torch.cat(out)
