"""The append to a paged cache (normalisation, rotation, page lookup) against its 64-bit form: head layouts, page
sizes, both cache types, ragged batches with empty sequences and rows of no sequence, and what it refuses to write.

Tolerances: the fp32 arithmetic of a normalised pair is off by less than 2^-20 of the two terms' magnitudes (a sum of
128 squares, a root, a division, four products: under 16 roundings of 2^-24), then one rounding: half a step, 2^-8
relative in bf16, 2^-4 in E4M3 (2^-10 absolute below its smallest normal)."""
import pytest
import torch

import nvfp4_weight_only_flint_b200 as fm
import paged_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _angles(n):
    inv = 10000.0 ** (-torch.arange(0, R.DH, 2, dtype=torch.float64) / R.DH)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    return [(torch.rand(R.DH, generator=g) + 0.5).to(torch.bfloat16) for _ in range(2)]


def _run(b, qw, kw, cs, rope, max_pos=None, status=None, k=None, v=None, q_out=None):
    c = b.cuda
    k = c(b.k).clone() if k is None else k
    v = c(b.v).clone() if v is None else v
    q_out = torch.full((b.T, b.hq, R.DH), 77.0, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
    fm.flint_qk_norm_rope_paged_kv(c(b.qkv), b.T, b.hq, b.hkv, c(qw), c(kw), c(cs) if rope else None,
                                   0 if not rope else (cs.shape[0] if max_pos is None else max_pos), rope, EPS,
                                   c(b.q_start), c(b.kv_len), b.B, c(b.table), b.max_pages, b.page, b.n_pages,
                                   b.dtype(), c(b.ks), c(b.vs), q_out, k, v, status)
    torch.cuda.synchronize()
    return q_out.cpu(), k.cpu(), v.cpu()


def _check(b, got, qw, kw, cs, rope, skip=()):
    (q, q_size), (k, k_size), v = R.append(b, qw, kw, cs, EPS, rope)
    q_out, kc, vc = got
    rows = [t for s in range(b.B) for t in range(int(b.q_start[s]), int(b.q_start[s + 1]))]
    assert ((q_out.double() - q).abs()[rows] <= 2 ** -8 * q.abs()[rows] + 2 ** -20 * q_size[rows]).all()
    others = [t for t in range(b.T) if t not in set(rows)]
    assert (q_out[others] == 77.0).all()  # rows of no sequence are left as they were
    touched = torch.zeros((b.n_pages, b.page), dtype=torch.bool)
    for s in range(b.B):
        for i in range(b.new[s]):
            t, p = int(b.q_start[s]) + i, b.kv[s] - b.new[s] + i
            if (s, p) in skip:
                continue
            page, row = int(b.table[s, p // b.page]), p % b.page
            touched[page, row] = True
            for got_row, ref, size, sc in ((kc, k[t], k_size[t], b.ks), (vc, v[t], v[t].abs(), b.vs)):
                g = got_row[page, row].float().double()
                if sc is None:
                    tol = 2 ** -8 * ref.abs() + 2 ** -20 * size
                else:
                    ref, size = ref / sc.double()[:, None], size / sc.double()[:, None]
                    ref = ref.clamp(-448, 448)
                    tol = 2 ** -4 * ref.abs() + 2 ** -10 + 2 ** -20 * size
                assert ((g - ref).abs() <= tol).all(), (s, p)
            if not b.e4m3:
                assert torch.equal(vc[page, row].view(torch.int16), b.qkv[t, b.hq + b.hkv:].view(torch.int16))
    for got_pool, was in ((kc, b.k), (vc, b.v)):  # every other cache row, bit for bit
        i = torch.uint8 if b.e4m3 else torch.int16
        assert torch.equal(got_pool.view(i)[~touched], was.view(i)[~touched])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,page", [(32, 4, 16), (7, 3, 32), (5, 1, 64), (1, 2, 128), (8, 8, 1024)])
def test_append_layouts(hq, hkv, page, e4m3):
    b = R.Paged(hq * 7 + page, [1, 0, 37, 5, 1], [1, 0, 37, 200, 129], hq, hkv, page, e4m3, pad=3)
    qw, kw = _weights(hq)
    cs = _angles(200)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(b, _run(b, qw, kw, cs, True, status=st), qw, kw, cs, True)
    assert int(st.item()) == 0


@pytest.mark.parametrize("norm,rope", [(False, False), (False, True), (True, False)])
def test_append_without_parts(norm, rope):
    b = R.Paged(3, [9, 2], [50, 2], 12, 4, 16)
    qw, kw = _weights(1) if norm else (None, None)
    cs = _angles(50)
    got = _run(b, qw, kw, cs, rope)
    _check(b, got, qw, kw, cs, rope)
    if not norm and not rope:  # nothing is computed: bits in, bits out
        assert torch.equal(got[0][:b.rows].view(torch.int16), b.qkv[:b.rows, :b.hq].view(torch.int16))


@pytest.mark.parametrize("B,T", [(1, 1), (1, 300), (17, 17), (300, 300), (1000, 1500)])
def test_append_finds_the_sequence(B, T):
    # the search over q_start, at batch sizes on both sides of its steps of 17, with empty sequences
    g = torch.Generator().manual_seed(B)
    cut = torch.sort(torch.randint(0, T + 1, (B - 1,), generator=g)).values.tolist()
    edges = [0] + cut + [T]
    new = [y - x for x, y in zip(edges, edges[1:])]
    kv = [n + int(torch.randint(0, 40, (1,), generator=g)) for n in new]
    b = R.Paged(B + 1, new, kv, 2, 1, 16)
    cs = _angles(max(kv))
    qw, kw = _weights(2)
    _check(b, _run(b, qw, kw, cs, True), qw, kw, cs, True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [511, 512, 513])
def test_append_call_sizes(T, e4m3):
    # two heads a half-warp up to 512 tokens, four above
    b = R.Paged(T, [T - 40, 40], [T, 77], 6, 1, 64, e4m3)
    cs = _angles(T)
    qw, kw = _weights(5)
    _check(b, _run(b, qw, kw, cs, True), qw, kw, cs, True)


def test_append_saturates_e4m3_and_large_values():
    b = R.Paged(5, [4], [4], 4, 2, 16, e4m3=True)
    b.qkv = b.qkv * 3000
    got = _run(b, None, None, None, False)
    _check(b, got, None, None, None, False)
    assert float(got[1].float().abs().nan_to_num(0).max()) == 448.0


@pytest.mark.parametrize("scale", [1.0, 3 / 128, 0.05, 7 / 64, 0.3])
def test_append_e4m3_codes_of_halfway_values(scale):
    # bf16 values over every binade that has codes, many halfway between two: the code is that of the fp32 quotient
    b = R.Paged(3, [16], [16], 4, 4, 16, e4m3=True)
    x = torch.arange(0x3800, 0x3800 + 16 * 4 * R.DH).to(torch.int16).view(torch.bfloat16).view(16, 4, R.DH)
    b.qkv[:, 4:8], b.qkv[:, 8:] = x, -x
    b.ks, b.vs = torch.full((4,), scale), torch.full((4,), scale)
    _, k, v = _run(b, None, None, None, False)
    want = (x.float() / torch.tensor(scale)).clamp(-448, 448)
    page = int(b.table[0, 0])
    assert torch.equal(k[page].view(torch.uint8), want.to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(v[page].view(torch.uint8), (-want).to(torch.float8_e4m3fn).view(torch.uint8))


def test_append_skips_what_has_no_place():
    b = R.Paged(8, [2, 3, 4, 1], [20, 40, 10, 33], 6, 2, 16, pad=1)
    b.table[1, 2] = b.n_pages          # positions 37..39 of sequence 1 have no page
    b.table[3, 2] = -1
    cs = _angles(60)
    qw, kw = _weights(3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(b, qw, kw, cs, True, status=st)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    _check(b, got, qw, kw, cs, True, skip={(1, 37), (1, 38), (1, 39), (3, 32)})
    # a length that cannot hold its new tokens, one past the block table, token rows outside the call
    for kv, q_start in (([20, 2, 10, 33], None), ([20, 40, 10, 16 * 3 + 1], None), (None, [0, 2, 5, 9, 90])):
        b2 = R.Paged(8, [2, 3, 4, 1], [20, 40, 10, 33], 6, 2, 16, pad=1)
        before = [x.clone() for x in (b2.k, b2.v)]
        if kv is not None:
            b2.kv_len = torch.tensor(kv, dtype=torch.int32)
        if q_start is not None:
            b2.q_start = torch.tensor(q_start, dtype=torch.int32)
        st.zero_()
        got = _run(b2, qw, kw, cs, True, status=st)
        assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
        s = 1 if kv and kv[1] == 2 else 3
        for pool, was in zip(got[1:], before):  # the sequence's own pages are as they were
            own = b2.table[s][b2.table[s] >= 0].long()
            assert torch.equal(pool[own].view(torch.int16), was[own].view(torch.int16))


def test_append_places_nothing_by_an_unsorted_q_start():
    # the search for a token's sequence may end at one that begins behind the token: no position, whatever lies in front
    # of the block table (here a page of the pool) and of the angles
    T, n_pages, max_pages = 64, 6, 2
    front = torch.full((64 + 2 * max_pages,), 3, dtype=torch.int32, device="cuda")
    table = front[64:].view(2, max_pages)
    table.copy_(torch.tensor([[0, 1], [2, 4]], dtype=torch.int32))
    cs = torch.cat([torch.full((T, R.DH), 7.0), _angles(64)]).cuda()[T:]
    qkv = torch.randn((T, 6, R.DH), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for q_start, kv in (([48, 49, 0], [1, 1]), ([63, 64, 0], [20, 20]), ([30, 34, 2], [4, 32])):
        k, v = (torch.full((n_pages, 16, 1, R.DH), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros((T, 4, R.DH), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        fm.flint_qk_norm_rope_paged_kv(qkv, T, 4, 1, None, None, cs, 64, True, EPS, i32(q_start), i32(kv), 2, table,
                                       max_pages, 16, n_pages, fm.FLINT_KV_BF16, None, None, q, k, v, st)
        torch.cuda.synchronize()
        assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
        assert (k == 5.0).all() and (v == 5.0).all()
        assert (q.abs() < 7.0).all()  # no angle from in front of the table


def test_append_position_past_the_angle_table():
    b = R.Paged(9, [3], [12], 4, 2, 16)
    cs = _angles(11)  # position 11 has no angles: appended unturned, flagged
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, _ = _run(b, None, None, cs, True, status=st)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    assert torch.equal(q[2], b.qkv[2, :4]) and torch.equal(k[b.table[0, 0], 11], b.qkv[2, 4:6])


def test_append_graph_replays_other_lengths_on_another_stream():
    b = R.Paged(10, [1, 1, 1], [30, 17, 64], 32, 4, 16, spare=9)
    cs, (qw, kw) = _angles(80), _weights(4)
    c = b.cuda
    dev = {n: c(getattr(b, n)) for n in ("qkv", "q_start", "kv_len", "table", "k", "v")}
    w = [c(qw), c(kw), c(cs)]
    q_out = torch.full((b.T, b.hq, R.DH), 77.0, dtype=torch.bfloat16, device="cuda")

    def call():
        fm.flint_qk_norm_rope_paged_kv(dev["qkv"], b.T, 32, 4, w[0], w[1], w[2], 80, True, EPS, dev["q_start"],
                                       dev["kv_len"], b.B, dev["table"], b.max_pages, 16, b.n_pages,
                                       fm.FLINT_KV_BF16, None, None, q_out, dev["k"], dev["v"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b2 = R.Paged(11, [1, 1, 1], [29, 18, 50], 32, 4, 16, spare=9)
    b2.max_pages, b2.n_pages = b.max_pages, b.n_pages
    table = torch.full((3, b.max_pages), -7, dtype=torch.int32)
    table[:, :b2.table.shape[1]] = b2.table
    b2.table = table
    pool = torch.zeros((b.n_pages, 16, 4, R.DH), dtype=torch.bfloat16)
    b2.k, b2.v = pool, pool.clone()
    for n in ("qkv", "kv_len", "table", "k", "v"):
        dev[n].copy_(getattr(b2, n))
    q_out.fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    _check(b2, (q_out.cpu(), dev["k"].cpu(), dev["v"].cpu()), qw, kw, cs, True)
