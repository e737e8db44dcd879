"""Attention of new tokens over the paged cache against its 64-bit form: decode and chunk calls, both cache types, head
layouts, page sizes, ragged and empty sequences, windows, rows of no sequence, lengths and pages that are invalid.
Everything the sequences do not own holds NaN. Bounds: paged_ref.check_attention."""
import pytest
import torch

import nvfp4_weight_only_flint_b200 as fm
import paged_ref as R

pytestmark = pytest.mark.gpu

DECODE = [([1], [1]), ([1], [17]), ([1], [4097]), ([1, 1, 1], [64, 65, 1000]), ([2, 1, 0, 2], [2, 300, 40, 129]),
          ([1] * 70, [3 + 29 * i for i in range(70)])]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_lengths(case, e4m3):
    new, kv = DECODE[case]
    b = R.Paged(100 + case, new, kv, 32, 4, 16, e4m3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.check_attention(R.run_attention(b, status=st), b, what=str((new[:4], kv[:4])))
    assert int(st.item()) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (3, 3, 32), (14, 2, 64), (16, 1, 128), (12, 4, 1024), (26, 2, 16)])
def test_decode_head_layouts(hq, hkv, page, e4m3):
    b = R.Paged(hq + page, [1, 1, 1], [5, 700, 130], hq, hkv, page, e4m3)
    R.check_attention(R.run_attention(b), b, what=f"{hq}/{hkv}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 15, 64, 700])
def test_decode_window(window, e4m3):
    b = R.Paged(window, [2, 1, 2], [2, 900, 333], 16, 2, 16, e4m3)
    R.check_attention(R.run_attention(b, window), b, window, what=f"window {window}")


@pytest.mark.parametrize("new", [[2, 1], [60, 40]])
def test_window_does_not_need_pages_in_front_of_it(new):
    # a sliding-window layer gives pages back: their table entries are no pages
    for e4m3 in (False, True):
        b = R.Paged(55, new, [700, 333], 8, 2, 16, e4m3)
        whole = R.attention(b, 100)
        for s in range(2):
            first = b.kv[s] - b.new[s] - 100 + 1  # first key any new token sees
            b.table[s, :first // 16] = -1
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = R.run_attention(b, 100, status=st)
        assert int(st.item()) == 0
        assert torch.equal(R.attention(b, 100), whole)
        R.check_attention(got, b, 100, what="freed pages")


def test_decode_peaked_scores():
    b = R.Paged(50, [1, 1], [3000, 200], q_gain=5.0)
    R.check_attention(R.run_attention(b), b, what="peaked")
    b = R.Paged(51, [1, 1], [3000, 200], q_gain=5.0, e4m3=True)
    R.check_attention(R.run_attention(b), b, what="peaked, e4m3")


def _invalid(new, kv, e4m3, hq=8, hkv=2):
    """What invalid lengths, rows and pages give, for a decode or a chunk call."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq = max(new)
    b = R.Paged(60, new, kv, hq, hkv, 16, e4m3, pad=2)
    got = R.run_attention(b, status=st, max_q=mq)
    assert int(st.item()) == 0
    R.check_attention(got, b)
    assert got[b.rows:].isnan().all()  # rows of no sequence keep the sentinel
    # a length below its new tokens, or past the block table: zeros, the others as before
    for bad in (new[1] - 1, -5, 16 * b.max_pages + 1, 2 ** 31 - 1):
        b = R.Paged(60, new, kv, hq, hkv, 16, e4m3, pad=2)
        b.kv_len[1] = bad
        st.zero_()
        out = R.run_attention(b, status=st, max_q=mq)
        assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
        r = slice(int(b.q_start[1]), int(b.q_start[2]))
        assert (out[r] == 0).all()
        out[r] = got[r]
        R.check_attention(out, b)
    # a page outside the pool counts as zero keys and values
    b = R.Paged(60, new, kv, hq, hkv, 16, e4m3, pad=2)
    b.table[2, 1], b.table[2, 3] = -1, b.n_pages
    st.zero_()
    out = R.run_attention(b, status=st, max_q=mq)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    R.check_attention(out, b)
    # token rows outside the call
    b = R.Paged(60, new, kv, hq, hkv, 16, e4m3, pad=2)
    b.q_start[-1] = b.T + 1
    st.zero_()
    out = R.run_attention(b, status=st, max_q=mq)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    last = slice(int(b.q_start[-2]), b.T)
    assert out[last].isnan().all()
    out[last] = got[last]
    R.check_attention(out, b)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_invalid(e4m3):
    _invalid([1, 2, 1, 2], [20, 50, 100, 33], e4m3)


def test_decode_more_tokens_than_announced():
    b = R.Paged(70, [1, 3, 1], [30, 30, 30], 8, 2, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = R.run_attention(b, status=st, max_q=2)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    assert (out[1:4] == 0).all()
    out[1:4] = R.attention(b)[1:4]
    R.check_attention(out, b)


def test_decode_split_is_the_same_in_every_run_and_graph():
    b = R.Paged(80, [1] * 5, [9000, 17, 4000, 1, 2500])
    c = b.cuda
    dev = [c(x) for x in (b.q, b.q_start, b.kv_len, b.table, b.k, b.v)]
    ws = torch.empty(fm.flint_paged_attention_workspace_bytes(b.T, b.B, 32, 4, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty((b.T, 32, R.DH), dtype=torch.bfloat16, device="cuda")

    def call(o=out, w=ws, stream=None):
        fm.flint_paged_attention(dev[0], b.T, dev[1], dev[2], b.B, dev[3], b.max_pages, 16, b.n_pages, dev[4], dev[5],
                                 fm.FLINT_KV_BF16, None, None, 32, 4, 1, 0, R.DH ** -0.5, o, w, stream=stream)
    call()
    torch.cuda.synchronize()
    first = out.clone()
    R.check_attention(first.cpu().double(), b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # the same graph with other lengths
    b.kv = [3000, 17, 1, 1, 2400]
    dev[2].copy_(torch.tensor(b.kv, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    R.check_attention(out.cpu().double(), b)
    # two calls at once, each with its own workspace
    side = torch.cuda.Stream()
    o2, w2 = torch.empty_like(out), torch.empty_like(ws)
    side.wait_stream(torch.cuda.current_stream())
    call()
    call(o2, w2, side)
    torch.cuda.synchronize()
    assert torch.equal(out, o2)


# 37 kv heads leave eight parts a head: sequences cut several times, parts of several sequences
LONG = [([1] * 5, [5000, 3333, 1, 64, 900], 0), ([8, 1, 5], [5000, 2500, 1500], 0), ([1], [8192], 0), ([1], [8128], 0),
        ([1, 2, 1], [9000, 4500, 7000], 4000), ([1] * 40, [37 + 11 * i for i in range(40)], 0)]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_decode_few_parts(case):
    new, kv, window = LONG[case]
    b = R.Paged(400 + case, new, kv, 74, 37, 32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.check_attention(R.run_attention(b, window, status=st), b, window, what=str((new[:4], kv[:4])))
    assert int(st.item()) == 0


def test_decode_other_lengths_in_the_same_tables():
    b = R.Paged(420, [1, 1, 1], [8000, 900, 300], 74, 37, 32)
    for kv in ([5, 70, 1], [1, 1, 1], [8000, 1, 200], [7800, 130, 300], [8000, 900, 300]):
        b.kv, b.kv_len = kv, torch.tensor(kv, dtype=torch.int32)
        R.check_attention(R.run_attention(b), b, what=str(kv))


CHUNK = [([17], [17]), ([1, 3], [1, 200]), ([128], [128]), ([300], [300]), ([40], [1000]), ([33, 1, 0, 150, 1], [33, 2000, 5, 700, 64]),
         ([5], [3001]), ([513, 700], [900, 701])]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(CHUNK)))
def test_chunk_lengths(case, e4m3):
    new, kv = CHUNK[case]
    b = R.Paged(200 + case, new, kv, 8, 1, 16, e4m3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.check_attention(R.run_attention(b, status=st), b, what=str((new, kv)))
    assert int(st.item()) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (3, 3, 32), (14, 2, 64), (16, 1, 128), (12, 4, 1024), (26, 2, 256),
                                         (32, 4, 64)])
def test_chunk_head_layouts(hq, hkv, page, e4m3):
    b = R.Paged(hq + page, [150, 1, 20], [150, 700, 333], hq, hkv, page, e4m3)
    R.check_attention(R.run_attention(b), b, what=f"{hq}/{hkv}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 100, 128, 700])
def test_chunk_window(window, e4m3):
    b = R.Paged(window, [200, 1, 50], [200, 900, 1333], 16, 2, 16, e4m3)
    R.check_attention(R.run_attention(b, window), b, window, what=f"window {window}")


def test_chunk_peaked_scores():
    # the running maximum moves by far more than the rescale threshold
    for e4m3 in (False, True):
        b = R.Paged(50, [70, 9], [2000, 200], 8, 1, q_gain=5.0, e4m3=e4m3)
        R.check_attention(R.run_attention(b), b, what=f"peaked, e4m3 {e4m3}")


@pytest.mark.parametrize("B,seed", [(1, 1), (40, 2), (200, 3)])
def test_chunk_many_sequences(B, seed):
    # parts that begin and end in every place of the line, sequences without tokens between
    g = torch.Generator().manual_seed(seed)
    new = [int(x) for x in torch.randint(0, 30 if B > 1 else 900, (B,), generator=g)]
    new[0] = max(new[0], 18)  # more than one register tile: the chunk kernel
    kv = [n + int(x) for n, x in zip(new, torch.randint(0, 300, (B,), generator=g))]
    b = R.Paged(seed, new, kv, 2, 2, 16)
    R.check_attention(R.run_attention(b), b, what=f"{B} sequences")


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_pairs_dealt_whole(e4m3):
    # many short pairs a CTA (150 kv heads: one CTA each), sequences without tokens between
    b = R.Paged(5, [300, 0, 70, 1, 0, 33], [310, 4, 90, 30, 0, 33], 150, 150, 16, e4m3)
    R.check_attention(R.run_attention(b), b, what="whole pairs")
    b = R.Paged(6, [1500], [1500], 74, 74, 64, e4m3)
    R.check_attention(R.run_attention(b), b, what="one prompt")


def test_chunk_more_kv_heads_than_parts():
    for hq, hkv in ((150, 150), (160, 80)):
        b = R.Paged(hq, [20, 17], [20, 150], hq, hkv, 16)
        R.check_attention(R.run_attention(b), b, what=f"{hq}/{hkv}")


def test_chunk_split_over_keys():
    # one short piece of a long sequence: its key tiles go to many CTAs and are joined
    for e4m3 in (False, True):
        b = R.Paged(90, [40, 2], [20_000, 9000], 16, 2, 64, e4m3)
        R.check_attention(R.run_attention(b), b, what=f"split, e4m3 {e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_invalid(e4m3):
    _invalid([20, 37, 3, 9], [20, 80, 100, 33], e4m3)


def test_chunk_more_tokens_than_announced():
    b = R.Paged(70, [20, 60, 1], [30, 90, 30], 8, 2, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = R.run_attention(b, status=st, max_q=40)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    assert (out[20:80] == 0).all()
    out[20:80] = R.attention(b)[20:80]
    R.check_attention(out, b)


def test_chunk_is_the_same_in_every_run_and_graph():
    b = R.Paged(80, [300, 17, 1, 90], [900, 17, 4000, 2500], 16, 2, 32)
    c = b.cuda
    dev = [c(x) for x in (b.q, b.q_start, b.kv_len, b.table, b.k, b.v)]
    ws = torch.empty(fm.flint_paged_attention_workspace_bytes(b.T, b.B, 16, 2, 300), dtype=torch.uint8, device="cuda")
    out = torch.empty((b.T, 16, R.DH), dtype=torch.bfloat16, device="cuda")

    def call(o=out, w=ws, stream=None):
        fm.flint_paged_attention(dev[0], b.T, dev[1], dev[2], b.B, dev[3], b.max_pages, 32, b.n_pages, dev[4], dev[5],
                                 fm.FLINT_KV_BF16, None, None, 16, 2, 300, 0, R.DH ** -0.5, o, w, stream=stream)
    call()
    torch.cuda.synchronize()
    first = out.clone()
    R.check_attention(first.cpu().double(), b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    b.kv = [880, 17, 1, 2400]
    dev[2].copy_(torch.tensor(b.kv, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    b.table = dev[3].cpu()
    R.check_attention(out.cpu().double(), b)
    side = torch.cuda.Stream()
    o2, w2 = torch.empty_like(out), torch.empty_like(ws)
    side.wait_stream(torch.cuda.current_stream())
    call()
    call(o2, w2, side)
    torch.cuda.synchronize()
    assert torch.equal(out, o2)


# finished by one part, cut into parts and joined by row or by head; tile pairs whole, cut, dealt
NAN_QUERY = [([1, 1, 1], [64, 65, 5000], 32, 4, 16), ([1] * 40, [3 + 100 * i for i in range(40)], 32, 4, 16),
             ([2, 1], [9, 300], 32, 4, 16), ([1], [9000], 8, 1, 16), ([300, 5], [300, 77], 8, 1, 16),
             ([40, 2], [20_000, 9000], 16, 2, 64), ([1500], [1500], 74, 74, 64)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(NAN_QUERY)))
def test_nan_in_a_query_stays_in_its_head(case, e4m3):
    new, kv, hq, hkv, page = NAN_QUERY[case]
    b = R.Paged(510 + case, new, kv, hq, hkv, page, e4m3)
    hit = [(0, hq - 1), (b.rows // 2, 0), (b.rows - 1, hq // 2)]
    clean = b.q.clone()
    for t, h in hit:
        b.q[t, h, 5] = float("nan")
    got = R.run_attention(b)
    b.q = clean
    ref = R.attention(b)
    for t, h in hit:
        assert got[t, h].isnan().all(), (t, h)
        got[t, h] = ref[t, h]
    R.check_attention(got, b, what="the other heads")


def _sink(seed, new, kv, hq, hkv, at):
    """An E4M3 batch in which one key outweighs each other one 2^22 to 2^24.5 times and has a zero value, as attention
    sinks do: the output is what the light keys leave. (The sink's key is along the queries, at a score of 16 nats =
    23.1 bits; the others' scores have a deviation of 0.2 nats.)"""
    b = R.Paged(seed, new, kv, hq, hkv, 16, e4m3=True)
    g = torch.Generator().manual_seed(seed + 1)
    base = torch.randn((hkv, R.DH), generator=g)
    b.q = base.repeat_interleave(hq // hkv, 0) + 0.02 * torch.randn((b.T, hq, R.DH), generator=g)
    b.q = b.q.to(torch.bfloat16)
    k = torch.randn((b.n_pages, b.page, hkv, R.DH), generator=g) * 0.2
    v = b.v.float()
    for s in range(b.B):
        p = at(kv[s])
        page, row = int(b.table[s, p // b.page]), p % b.page
        k[page, row] = base * (16.0 * R.DH ** 0.5 / base.square().sum(-1, keepdim=True))
        v[page, row] = 0.0
    k = (k / b.ks[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    v = v.to(torch.float8_e4m3fn).view(torch.uint8)
    k[~b.live], v[~b.live] = 0x7F, 0x7F
    b.k, b.v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return b


@pytest.mark.parametrize("new,kv", [([1, 1], [3000, 200]), ([2, 1], [700, 9000]), ([70, 9], [2000, 200]),
                                    ([300], [700])])
@pytest.mark.parametrize("at", ["first", "middle"])
def test_light_keys_behind_a_heavy_one(new, kv, at):
    # their weights have to keep f16's 11 bits (check_attention's bound), 2^-24.5 of the largest as they are
    b = _sink(500, new, kv, 8, 2, (lambda n: 0) if at == "first" else (lambda n: n // 2))
    R.check_attention(R.run_attention(b), b, what=f"{at} key")


@pytest.mark.parametrize("new,kv", [([1, 2], [700, 90]), ([150, 1, 20], [150, 700, 333])])
def test_windows_past_every_position(new, kv):
    # up to the largest int: the same as no window, bit for bit
    for e4m3 in (False, True):
        b = R.Paged(530, new, kv, 8, 2, 16, e4m3)
        whole = R.run_attention(b)
        R.check_attention(whole, b)
        for window in (2 ** 30, 2 ** 31 - 1):
            assert torch.equal(R.run_attention(b, window), whole)
        R.check_attention(R.run_attention(b, 2 ** 30 - 1), b)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv", [75, 148, 297])
def test_one_part_a_kv_head(hkv, e4m3):
    # nothing is cut, and the workspace holds no partials
    for new, kv in (([1, 2, 0], [900, 70, 3]), ([40, 3], [300, 150])):
        b = R.Paged(hkv, new, kv, hkv, hkv, 16, e4m3)
        nb = fm.flint_paged_attention_workspace_bytes(b.T, b.B, hkv, hkv, max(new))
        if hkv > 148:
            assert nb < 1e5
        behind = torch.full((nb + 4096,), 0x55, dtype=torch.uint8, device="cuda")
        R.check_attention(R.run_attention(b, ws=behind), b, what=f"{hkv} kv heads")
        assert (behind[nb:] == 0x55).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,kv", [([384] * 4, [1084, 384, 1084, 384]), ([128] * 12, [228] * 12),
                                    ([100] * 10, [1600, 100, 100, 1600, 1600, 100, 100, 1600, 1600, 100])])
def test_chunk_pairs_dealt_or_cut(new, kv, e4m3):
    # two CTAs a kv head, ten or twelve tile pairs: dealt whole in the first two batches, cut in the last, whose long
    # pairs would all go to one CTA
    b = R.Paged(540 + len(new), new, kv, 148, 74, 64, e4m3)
    R.check_attention(R.run_attention(b), b, what=str((new[:4], kv[:4])))


@pytest.mark.parametrize("max_q", [1, 40])
def test_steps_without_any_token_write_nothing(max_q):
    for e4m3 in (False, True):
        b = R.Paged(550, [0, 0, 0], [5, 900, 0], 8, 2, 16, e4m3, pad=3)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        for start in ([0, 0, 0, 0], [2, 2, 2, 2], [3, 3, 3, 3]):
            b.q_start = torch.tensor(start, dtype=torch.int32)
            assert R.run_attention(b, max_q=max_q, status=st).isnan().all()
        assert int(st.item()) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_unsorted_q_start_stays_within_the_call(e4m3):
    # sequences that begin behind their ends, or share rows, are flagged or race for their rows; nothing else is touched
    for max_q in (2, 40):
        b = R.Paged(560, [2, 2, 2], [60, 60, 60], 8, 2, 16, e4m3, pad=4)
        for start in ([4, 6, 0, 2], [6, 0, 2, 1], [0, 2, -5, 2], [2, 2 ** 31 - 1, 0, 2], [-2 ** 31, 0, 1, 2]):
            b.q_start = torch.tensor(start, dtype=torch.int32)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = R.run_attention(b, max_q=max_q, status=st)
            assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
            owned = {t for x, y in zip(start, start[1:]) if 0 <= x <= y <= b.T for t in range(x, y)}
            for t in range(b.T):
                assert out[t].isnan().all() == (t not in owned), (start, t)
