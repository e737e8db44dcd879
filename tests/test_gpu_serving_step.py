"""A serving step as it is used: append the batch's new tokens to the paged cache, attend over it, the MoE layer, the
output head, sample; a prompt call, then decode steps that feed on it, each checked stage by stage against the 64-bit
forms on what the stage before produced; and the whole decode step as one captured graph, replayed with other lengths."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_flint_b200 as fm
import paged_ref as R
import synth
from gpu_layer import GpuLayer

pytestmark = pytest.mark.gpu

HQ, HKV, DH, PAGE, D, V = 4, 1, 128, 16, 512, 5000  # 4 x 128 = the layer's 512


class Step:
    """Buffers of a batch of B sequences over a pool, as a serving loop keeps them."""

    def __init__(self, B, max_len, T, e4m3):
        self.B, self.T, self.e4m3, self.max_pages = B, T, e4m3, -(-max_len // PAGE)
        self.n_pages = B * self.max_pages + 2
        g = torch.Generator().manual_seed(3)
        order = torch.randperm(self.n_pages, generator=g)[:B * self.max_pages].to(torch.int32)
        self.table = order.view(B, self.max_pages).cuda()
        dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        shape = (self.n_pages, PAGE, HKV, DH)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.float32).to(dt).cuda() for _ in range(2))
        self.scales = [torch.tensor([0.03], device="cuda"), torch.tensor([0.02], device="cuda")] if e4m3 else [None, None]
        inv = 10000.0 ** (-torch.arange(0, DH, 2, dtype=torch.float64) / DH)
        a = torch.arange(max_len, dtype=torch.float64)[:, None] * inv
        self.cs, self.max_len = torch.cat([a.cos(), a.sin()], 1).float().cuda(), max_len
        self.w = [(torch.rand(DH, generator=g) + 0.5).to(torch.bfloat16).cuda() for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.layer = GpuLayer(synth.CONFIGS["cfg0"], seed=1, max_tokens=8)
        self.router = torch.from_numpy(synth.make_router(synth.CONFIGS["cfg0"], 1, synth.x_bits(1, 4, D)).view(
            np.int16)).cuda()
        head = torch.randn((V, D), generator=g) * 0.2
        self.head = [torch.empty((V, D // 2), dtype=torch.uint8, device="cuda"),
                     torch.empty((V, D // 16), dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")]
        self.ws_head = torch.zeros(2048, dtype=torch.uint8, device="cuda")
        fm.flint_pack_nvfp4_dense(head.cuda(), 0, V, D, *self.head, self.ws_head)
        self.calls = {}

    def buffers(self, T, max_q):
        if T not in self.calls:
            e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
            nb = fm.flint_paged_attention_workspace_bytes(T, self.B, HQ, HKV, max_q)
            self.calls[T] = {"q": e(T, HQ, DH), "att": e(T, HQ, DH), "moe": e(self.B, D), "logits": e(self.B, V, dt=torch.float32),
                             "ws": e(nb, dt=torch.uint8), "tok": e(self.B, dt=torch.int32), "lp": e(self.B, dt=torch.float32)}
        return self.calls[T]

    def run(self, qkv, q_start, kv_len, T, max_q, last, temperature, top_k, top_p, u):
        b = self.buffers(T, max_q)
        dt = fm.FLINT_KV_E4M3 if self.e4m3 else fm.FLINT_KV_BF16
        fm.flint_qk_norm_rope_paged_kv(qkv, T, HQ, HKV, *self.w, self.cs, self.max_len, True, 1e-6, q_start, kv_len,
                                       self.B, self.table, self.max_pages, PAGE, self.n_pages, dt, *self.scales, b["q"],
                                       self.k, self.v, self.status)
        fm.flint_paged_attention(b["q"], T, q_start, kv_len, self.B, self.table, self.max_pages, PAGE, self.n_pages,
                                 self.k, self.v, dt, *self.scales, HQ, HKV, max_q, 0, DH ** -0.5, b["att"], b["ws"],
                                 self.status)
        x = b["att"].view(T, D).index_select(0, last)  # the last new token of each sequence
        fm.flint_moe_forward(x, self.B, self.router, self.layer.weights, self.layer.shape, x, b["moe"], self.layer.ws)
        fm.flint_lm_head(b["moe"], self.B, *self.head, V, D, b["logits"], self.ws_head)
        fm.flint_sample(b["logits"], self.B, V, V, fm.FLINT_LOGITS_F32, temperature, top_k, top_p, None, u, b["tok"],
                        b["lp"], self.status)
        return b


def _check(s, b, qkv, new, kv, keep, params):
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    ref = R.Paged(0, new, kv, HQ, HKV, PAGE, s.e4m3)
    ref.table, ref.max_pages, ref.n_pages, ref.qkv = s.table.cpu(), s.max_pages, s.n_pages, qkv.cpu()
    ref.k, ref.v = s.k.cpu(), s.v.cpu()
    if s.e4m3:
        ref.ks, ref.vs = s.scales[0].cpu(), s.scales[1].cpu()
    (q, qs), (k, ks_), v = R.append(ref, s.w[0].cpu(), s.w[1].cpu(), s.cs.cpu(), 1e-6, True)
    assert ((b["q"].cpu().double() - q).abs() <= 2 ** -8 * q.abs() + 2 ** -20 * qs).all()
    half = 2 ** -4 if s.e4m3 else 2 ** -8
    for i in range(len(new)):  # the appended rows, and earlier calls' rows untouched
        kk, vv = ref.values(i)
        r0 = int(ref.q_start[i])
        rows = slice(kv[i] - new[i], kv[i])
        sc = s.scales[0].cpu().double() if s.e4m3 else 1.0
        assert ((kk[rows] - k[r0:r0 + new[i]]).abs() <= half * k[r0:r0 + new[i]].abs() + 2 ** -10 * sc +
                2 ** -20 * ks_[r0:r0 + new[i]]).all()
        if i in keep:
            assert torch.equal(kk[:keep[i][0].shape[0]], keep[i][0]) and torch.equal(vv[:keep[i][1].shape[0]], keep[i][1])
        keep[i] = (kk, vv)
    ref.q = b["q"].cpu()
    R.check_attention(b["att"].cpu().double(), ref, what="attention of the step")
    logits = b["logits"].cpu().double()
    f32 = lambda x: float(x)  # noqa: E731
    for i in range(len(new)):
        want, lw = R.sample(logits[i], f32(params[0][i]), int(params[1][i]), f32(params[2][i]), 0.0, f32(params[3][i]))
        assert int(b["tok"][i]) == want
        assert abs(float(b["lp"][i]) - lw) <= 2 ** -23 * abs(lw) + 2 ** -26


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_steps(e4m3):
    B, prompts = 4, [37, 5, 64, 1]
    s = Step(B, 120, sum(prompts), e4m3)
    g = torch.Generator().manual_seed(7)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    params = [torch.tensor([1.0, 0.7, 0.0, 1.3]).cuda(), i32([0, 50, 0, 0]), torch.tensor([0.9, 1.0, 1.0, 0.95]).cuda(), None]
    qkv_of = lambda T: torch.randn((T, HQ + 2 * HKV, DH), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    keep, kv = {}, list(prompts)
    starts = [sum(prompts[:i]) for i in range(B + 1)]
    qkv = qkv_of(sum(prompts))
    params[3] = torch.rand(B, generator=g).cuda()
    b = s.run(qkv, i32(starts), i32(kv), sum(prompts), max(prompts), i32([x - 1 for x in starts[1:]]).long(), *params)
    _check(s, b, qkv, prompts, kv, keep, params)
    # decode steps as one captured graph: fixed buffers, new contents
    q_start, kv_len, last = i32(list(range(B + 1))), i32(kv), torch.arange(B, device="cuda")
    qkv = qkv_of(B)
    call = lambda: s.run(qkv, q_start, kv_len, B, 1, last, *params)  # noqa: E731
    kv_len.copy_(i32([x + 1 for x in kv]))
    call()  # warm-up: appends the same rows that the first replay appends
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = call()
    for _ in range(3):
        kv = [x + 1 for x in kv]
        kv_len.copy_(i32(kv))
        qkv.copy_(qkv_of(B))
        params[3].copy_(torch.rand(B, generator=g).cuda())
        graph.replay()
        _check(s, b, qkv, [1] * B, kv, keep, params)


def test_other_threads_run_while_a_launch_waits():
    """A launch into a full queue waits for the GPU, without the interpreter lock."""
    import threading
    import time
    x, u = torch.zeros((1, 100), device="cuda"), torch.zeros(1, device="cuda")
    tok = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: fm.flint_sample(x, 1, 100, 100, fm.FLINT_LOGITS_F32, None, None, None, None, u, tok)  # noqa: E731
    call()
    torch.cuda.synchronize()
    gap, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0], last = max(gap[0], now - last), now

    other = threading.Thread(target=tick)
    other.start()
    torch.cuda._sleep(1_000_000_000)  # half a second: more launches behind it than the queue holds
    longest = 0.0
    for _ in range(3000):
        t = time.perf_counter()
        call()
        longest = max(longest, time.perf_counter() - t)
    stop.set()
    other.join()
    torch.cuda.synchronize()
    assert longest < 0.1 or gap[0] < longest / 2, (longest, gap[0])
