"""Plain 64-bit forms of the paged serving operators (torch double, one sequence and one row at a time) and builders of
small paged batches for their tests."""
import math

import torch

import nvfp4_weight_only_flint_b200 as fm

DH = 128


class Paged:
    """A batch of sequences with `new[s]` new tokens and `kv[s]` cached positions (new ones included) over a shuffled
    pool. Rows of the pool that belong to no position hold NaN (bf16) or the NaN code (E4M3)."""

    def __init__(self, seed, new, kv, hq=32, hkv=4, page=16, e4m3=False, pad=0, spare=3, v_gain=1.0, q_gain=1.0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.hq, self.hkv, self.page, self.e4m3 = list(new), list(kv), hq, hkv, page, e4m3
        self.B, self.rows = len(new), sum(new)
        self.T = self.rows + pad
        used = [-(-x // page) for x in kv]
        self.max_pages = max(used + [1])
        self.n_pages = sum(used) + spare
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)  # unused entries are not pages
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.q_start = torch.tensor([sum(new[:i]) for i in range(self.B + 1)], dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32)
        self.q = (torch.randn((self.T, hq, DH), generator=g) * q_gain).to(torch.bfloat16)
        self.qkv = torch.randn((self.T, hq + 2 * hkv, DH), generator=g).to(torch.bfloat16)
        k = torch.randn((self.n_pages, page, hkv, DH), generator=g)
        v = torch.randn((self.n_pages, page, hkv, DH), generator=g) * v_gain
        self.ks = (torch.rand(hkv, generator=g) * 0.02 + 0.02) if e4m3 else None
        self.vs = (torch.rand(hkv, generator=g) * 0.02 + 0.01) if e4m3 else None
        live = torch.zeros((self.n_pages, page), dtype=torch.bool)
        for s in range(self.B):
            for p in range(self.kv[s]):
                live[self.table[s, p // page], p % page] = True
        if e4m3:
            to8 = lambda x, sc: (x / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
            k, v = to8(k, self.ks), to8(v, self.vs)
            k[~live], v[~live] = 0x7F, 0x7F
            self.k, self.v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        else:
            k[~live], v[~live] = math.nan, math.nan
            self.k, self.v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        self.live = live
        self.device = device

    def dtype(self):
        return fm.FLINT_KV_E4M3 if self.e4m3 else fm.FLINT_KV_BF16

    def cuda(self, x):
        return None if x is None else x.to(self.device)

    def values(self, s):
        """Keys and values of sequence s in double, [kv][hkv][128]; a page outside the pool reads as zeros."""
        out = []
        for pool, sc in ((self.k, self.ks), (self.v, self.vs)):
            x = pool.to(torch.float32).double()
            if sc is not None:
                x = x * sc.double()[:, None]
            rows = []
            for p in range(self.kv[s]):
                page = int(self.table[s, p // self.page])
                rows.append(x[page, p % self.page] if 0 <= page < self.n_pages else torch.zeros(self.hkv, DH).double())
            out.append(torch.stack(rows) if rows else torch.zeros(0, self.hkv, DH).double())
        return out


def attention(b, window=0, scale=DH ** -0.5, abs_values=False):
    """Each token's output in double, [T][hq][128]; zeros for rows of no sequence. abs_values: over |v|."""
    out = torch.zeros((b.T, b.hq, DH), dtype=torch.float64)
    group = b.hq // b.hkv
    for s in range(b.B):
        n, kv, r0 = b.new[s], b.kv[s], int(b.q_start[s])
        if n == 0:
            continue
        k, v = b.values(s)
        v = v.abs() if abs_values else v
        q = b.q[r0:r0 + n].double().view(n, b.hkv, group, DH)
        x = torch.einsum("nhgd,jhd->hgnj", q, k) * scale
        pos, j = torch.arange(kv - n, kv)[:, None], torch.arange(kv)[None, :]
        sees = j <= pos
        if window > 0:
            sees &= j > pos - window
        w = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
        out[r0:r0 + n] = torch.einsum("hgnj,jhd->nhgd", w, v).reshape(n, b.hq, DH)
    return out


def run_attention(b, window=0, scale=DH ** -0.5, status=None, max_q=None, fill=float("nan"), stream=None, ws=None):
    """The operator's output, on the CPU as double; unwritten rows keep `fill`."""
    max_q = max(b.new + [1]) if max_q is None else max_q
    out = torch.full((b.T, b.hq, DH), fill, dtype=torch.bfloat16, device=b.device)
    if ws is None:
        nb = fm.flint_paged_attention_workspace_bytes(b.T, b.B, b.hq, b.hkv, max_q)
        ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device=b.device)  # NaN partials
    c = b.cuda
    fm.flint_paged_attention(c(b.q), b.T, c(b.q_start), c(b.kv_len), b.B, c(b.table), b.max_pages, b.page, b.n_pages,
                             c(b.k), c(b.v), b.dtype(), c(b.ks), c(b.vs), b.hq, b.hkv, max_q, window, scale, out, ws,
                             status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().double()


def check_attention(got, b, window=0, scale=DH ** -0.5, what=""):
    """Bounds, with u the half step of a rounding (bf16 2^-8, f16 2^-11): each weight enters the value sum rounded once
    (relative u), the sum of the rounded weights divides it (another u), so the output is off by at most 2 u A (1 +
    2u), A = sum_j w_j |v_j|; fp32 scores, exponentials (2^-22) and sums add less than 2^-12 A at the scores of these
    tests (|score| < 100: 100 * 2^-22 and 128 products of relative 2^-24); the output's own rounding is 2^-8 of it."""
    ref = attention(b, window, scale)
    a = attention(b, window, scale, abs_values=True)
    u = 2.0 ** -11 if b.e4m3 else 2.0 ** -8
    tol = 2.0 ** -8 * ref.abs() + (2 * u * (1 + 2 * u) + 2.0 ** -12) * a + 1e-30
    rows = slice(0, b.rows)
    err = (got - ref).abs()[rows]
    bad = ~(err <= tol[rows])
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol[rows]).nan_to_num(1e9).max()):.3g} of the bound"


def append(b, qw, kw, cos_sin, eps, rope):
    """(q [T][hq][128], k [T][hkv][128] and v as stored values before rounding, magnitude of the terms of q and k)."""
    x = b.qkv.double()
    q, k, v = x[:, :b.hq], x[:, b.hq:b.hq + b.hkv], x[:, b.hq + b.hkv:]
    out = []
    pos = torch.zeros(b.T, dtype=torch.long)
    for s in range(b.B):
        r0 = int(b.q_start[s])
        pos[r0:r0 + b.new[s]] = torch.arange(b.kv[s] - b.new[s], b.kv[s])
    for y, w in ((q, qw), (k, kw)):
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
        size = y.abs() + torch.cat([y[..., 64:], y[..., :64]], -1).abs()
        if rope:
            c, s_ = cos_sin[pos].double()[:, None, :64], cos_sin[pos].double()[:, None, 64:]
            y = torch.cat([y[..., :64] * c - y[..., 64:] * s_, y[..., 64:] * c + y[..., :64] * s_], -1)
        out.append((y, size))
    return out[0], out[1], v


def sample(x, t, k, p, m, u):
    """One row: (token, log-probability); x double [V]."""
    x = x.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    top = float(x.max())
    if top == -math.inf:
        return -1, -math.inf
    if t == 0:
        return int(torch.nonzero(x == x.max())[0, 0]), 0.0
    w = torch.where(x == x.max(), 1.0, torch.exp((x - top) / t))
    w[x == -math.inf] = 0.0
    order = torch.argsort(x, descending=True, stable=True)
    if 0 < k < x.numel():
        order = order[:k]
    if p < 1:
        ws = w[order]
        before = torch.cat([torch.zeros(1).double(), torch.cumsum(ws, 0)[:-1]])
        keep = before < p * ws.sum()
        keep[0] = True
        order = order[keep]
    kept = torch.sort(order).values
    kept = kept[w[kept] >= min(m, 1.0)]
    c = torch.cumsum(w[kept], 0)
    i = int(torch.nonzero(c > u * c[-1])[0, 0])
    return int(kept[i]), math.log(float(w[kept[i]] / c[-1]))
