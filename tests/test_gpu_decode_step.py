"""The decode-side operators together, as a decoder's attention block runs them: packed query, key and value
projections, adapters on them, rotary positions, the write into the KV8 cache, attention over it and the output
projection with its adapters.  Each call is checked against its definition for the operands it received; a captured
step replays the following tokens with the eager steps' bits; another stream with buffers of its own runs beside it."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from parity_util import check_float, host
from test_gpu_kv8 import check_attention, i32, starts
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu

HQ, HK, D, P, RANK, L = 8, 2, 64, 32, 16, 3
HIDDEN = HQ * D
BASE = 500000.0


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


class Block:
    def __init__(self, lb, seed, n_seqs, max_rows, max_pages):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape, scale):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.lb, self.w, self.a, self.b = lb, {}, {}, {}
        for name, n in (("q", HQ * D), ("k", HK * D), ("v", HK * D), ("o", HIDDEN)):
            q = torch.empty((n, HIDDEN // 2), dtype=torch.uint8, device="cuda")
            s = torch.empty((n, HIDDEN // 64), dtype=torch.int16, device="cuda")
            lb.lowbit_quantize("int4", randn(n, HIDDEN, scale=HIDDEN ** -0.5), q, s)
            self.w[name] = q, s
            self.a[name] = randn(L, RANK, HIDDEN, scale=HIDDEN ** -0.5).bfloat16()
            self.b[name] = randn(L, n, RANK, scale=0.3 * RANK ** -0.5).bfloat16()
        self.ranks, self.scales = i32([16, 8, 3]), torch.tensor([1.0, -0.5, 2.0], device="cuda")
        self.phases = lb.lowbit_rope_phases(D, BASE).cuda()
        n_pages = n_seqs * max_pages + 1
        self.cache = lb.KV8Cache.empty(n_pages, HK, P, D)
        order = np.random.default_rng(seed).permutation(n_pages - 1)
        self.table = order.reshape(n_seqs, max_pages).astype(np.int32)
        self.dtable = i32(self.table)
        n = max(lb.lowbit_lora_workspace_bytes(2, max_rows, HIDDEN, HIDDEN, RANK), 16)
        self.lora_ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        n = lb.lowbit_kv8_attention_workspace_bytes(self.cache, n_seqs, max_rows, HQ)
        self.attn_ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def lora(self, x, ids, names, base, y):
        self.lb.lowbit_lora_add_group(x, ids, [self.a[n] for n in names], [self.b[n] for n in names], base, y,
                                      ranks=self.ranks, scales=self.scales, workspace=self.lora_ws)

    def project(self, names, x, ys):
        # 32 rows at a time: with more, the int4 product adds slices of K in no fixed order, and a run's last bits
        # would differ from the next one's before the calls compared here
        for m in range(0, x.shape[0], 32):
            self.lb.lowbit_int4g64_gemm_group([self.w[n][0] for n in names], [self.w[n][1] for n in names], x[m:m + 32],
                                              [y[m:m + 32] for y in ys])

    def step(self, x, ids, positions, lens, row_start=None, keep=False):
        """x bf16 [T][HIDDEN] -> fp32 [T][HIDDEN], and what each call received and gave."""
        lb, T = self.lb, x.shape[0]
        new = lambda n, dtype=torch.float32: torch.empty((T, n), dtype=dtype, device="cuda")
        q, k, v, o = new(HQ * D), new(HK * D), new(HK * D), new(HIDDEN)
        self.project(["q"], x, [q])
        self.project(["k", "v"], x, [k, v])
        shared = [t.clone() for t in (q, k, v)] if keep else None
        self.lora(x, ids, ["q"], [q], [q])
        self.lora(x, ids, ["k", "v"], [k, v], [k, v])
        q3, k3, v3 = q.view(T, HQ, D), k.view(T, HK, D), v.view(T, HK, D)
        qr, kr = new(HQ * D, torch.bfloat16).view(T, HQ, D), new(HK * D, torch.bfloat16).view(T, HK, D)
        lb.lowbit_rope(q3, qr, k3, kr, positions, self.phases)
        before = [host(t).copy() for t in (self.cache.k, self.cache.k_scales, self.cache.v, self.cache.v_scales)] if keep else None
        lb.lowbit_kv8_append(self.cache, self.dtable, lens, kr, v3, row_start=row_start)
        att = new(HQ * D, torch.bfloat16).view(T, HQ, D)
        lb.lowbit_kv8_attention(self.cache, self.dtable, lens, qr, att, D ** -0.5, row_start=row_start, workspace=self.attn_ws)
        self.project(["o"], att.view(T, HIDDEN), [o])
        first = o.clone() if keep else None
        self.lora(att.view(T, HIDDEN), ids, ["o"], [o], [o])
        return o, dict(shared=shared, qkv=(q, k, v), rope=(qr, kr), before=before, att=att, o=first) if keep else None

    def check(self, x, ids, positions, lens, row_start, o, rec):
        def lora(name, x, base, y):
            want, ab = ref.lora(ref.bf16_to_f64(x), host(ids), ref.bf16_to_f64(self.a[name]), ref.bf16_to_f64(self.b[name]),
                                host(base).astype(np.float64), host(self.ranks), host(self.scales))
            check_float(host(y), want, ab, name)

        for name, base, y in zip("qkv", rec["shared"], rec["qkv"]):
            lora(name, x, base, y)
        T = x.shape[0]
        freq = [BASE ** (-2.0 * j / D) for j in range(D // 2)]
        q, k, v = (t.view(T, -1, D) for t in rec["qkv"])
        check_rope(rec["rope"][0], q, positions, freq, False, 1.0)
        check_rope(rec["rope"][1], k, positions, freq, False, 1.0)
        lens, rs, c = host(lens), None if row_start is None else host(row_start), self.cache
        for i, (t, codes, scales) in enumerate(((rec["rope"][1], c.k, c.k_scales), (v, c.v, c.v_scales))):
            wc, ws = ref.append(rec["before"][2 * i], rec["before"][2 * i + 1], t.float().cpu().numpy(), lens, self.table, rs)
            assert np.array_equal(host(codes), wc) and np.array_equal(host(scales), ws)
        check_attention(c, self.table, lens, rec["rope"][0], D ** -0.5, rs, rec["att"])
        lora("o", rec["att"].view(T, HIDDEN), rec["o"], o)


def tokens(seed, T):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, HIDDEN), generator=g, device="cuda").bfloat16()


ROWS = [5, 70, 0, 33]  # the third sequence is an idle slot


def prompt(block, seed, keep):
    rs = starts(ROWS)
    ids = i32([i for i, n in zip([0, 2, 1, -1], ROWS) for _ in range(n)])
    positions = i32([p for n in ROWS for p in range(n)])
    args = tokens(seed, sum(ROWS)), ids, positions, i32(ROWS), i32(rs)
    o, rec = block.step(*args, keep=keep)
    if keep:
        block.check(*args, o, rec)
    return o


def test_prompt_then_tokens(lb):
    block = Block(lb, 1, 4, sum(ROWS), 4)
    prompt(block, 10, keep=True)
    for t in range(3):
        lens = [n + t + 1 if n else 0 for n in ROWS]
        args = tokens(20 + t, 4), i32([0, 2, -1, 1]), i32([max(n - 1, 0) for n in lens]), i32(lens), None
        o, rec = block.step(*args, keep=True)
        block.check(*args, o, rec)
        assert (rec["att"][2] == 0).all()
    # four proposed tokens a sequence at once
    lens = [n + 7 if n else 0 for n in ROWS]
    rs = starts([4 if n else 0 for n in ROWS])
    pos = [p for n in lens for p in range(n - 4, n) if n]
    args = tokens(30, 12), i32([0] * 4 + [2] * 4 + [1] * 4), i32(pos), i32(lens), i32(rs)
    o, rec = block.step(*args, keep=True)
    block.check(*args, o, rec)
    assert lb.lowbit_fault_flags() == 0


def test_captured_step_and_a_second_stream(lb):
    steps = 40  # over a page's end for every sequence
    x, ids = tokens(5, 4), i32([0, 2, -1, 1])
    position, lens = i32([0] * 4), i32([0] * 4)

    def advance(t):
        now = [n + t + 1 if n else 0 for n in ROWS]
        x.copy_(tokens(100 + t, 4))
        position.copy_(i32([max(n - 1, 0) for n in now]))
        lens.copy_(i32(now))

    eager, replayed = Block(lb, 2, 4, sum(ROWS), 4), Block(lb, 2, 4, sum(ROWS), 4)
    want = [prompt(eager, 11, keep=False)]
    got = [prompt(replayed, 11, keep=False)]
    assert torch.equal(want[0], got[0])
    for t in range(steps):
        advance(t)
        want.append(eager.step(x, ids, position, lens)[0])
    advance(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = replayed.step(x, ids, position, lens)
    # beside the replays, a block of its own buffers on another stream
    other, side = Block(lb, 3, 4, sum(ROWS), 4), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        beside = [prompt(other, 12, keep=False) for _ in range(4)]
    for t in range(steps):
        advance(t)
        graph.replay()
        got.append(out.clone())
    with torch.cuda.stream(side):
        beside += [prompt(other, 12, keep=False) for _ in range(4)]
    torch.cuda.synchronize()
    for t, (w, g) in enumerate(zip(want, got)):
        assert torch.equal(w, g), f"step {t}"
    for b in beside[1:]:
        assert torch.equal(b, beside[0])
    for name in ("k", "k_scales", "v", "v_scales"):
        assert torch.equal(getattr(eager.cache, name), getattr(replayed.cache, name))
    assert lb.lowbit_fault_flags() == 0


def test_workspaces_of_another_kind_are_refused(lb):
    block = Block(lb, 4, 1, 4, 1)
    x, ids, y = tokens(1, 4), i32([0, 1, 2, 0]), torch.zeros((4, HIDDEN), device="cuda")
    att = torch.zeros((1, HQ, D), dtype=torch.bfloat16, device="cuda")
    for wrong in (lambda t: t.cpu(), lambda t: t.repeat(2)[::2]):
        with pytest.raises(ValueError):
            lb.lowbit_lora_add(x, ids, block.a["q"], block.b["q"], y, y, workspace=wrong(block.lora_ws))
        with pytest.raises(ValueError):
            lb.lowbit_kv8_attention(block.cache, block.dtable, i32([1]), att, att, 1.0, workspace=wrong(block.attn_ws))
