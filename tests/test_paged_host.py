"""Host-side checks of the paged serving operators: bad arguments are refused before anything is launched, and empty
calls are no-ops (no GPU needed: the pointers below are never dereferenced)."""
import pytest

import nvfp4_weight_only_flint_b200 as fm
from nvfp4_weight_only_flint_b200 import build as fbuild

A = 0x100000


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fm.lib()


BATCH = dict(T=4, B=2, mp=8, page=16, pages=64, dt=0, ks=None, vs=None, qs=A, kl=A, bt=A, k=A, v=A, dh=128, hq=32,
             hkv=4)
BAD_BATCH = [(dict(page=8), -2), (dict(page=24), -2), (dict(page=2048), -2), (dict(dt=2), -1), (dict(T=-1), -1),
             (dict(B=-1), -1), (dict(mp=-1), -1), (dict(pages=-1), -1), (dict(pages=1 << 27), -2), (dict(qs=None), -1),
             (dict(kl=None), -1), (dict(bt=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(dt=1), -1),
             (dict(dt=1, ks=A), -1), (dict(k=A + 8), -3), (dict(v=A + 2), -3), (dict(qs=A + 2), -3),
             (dict(dt=1, ks=A, vs=A + 1), -3), (dict(dh=64), -2), (dict(hq=0), -1), (dict(hkv=0), -1)]


def _append(L, qkv=A, qw=A, kw=A, cs=A, max_pos=16, rope=1, eps=1e-6, q_out=A, **kw2):
    b = {**BATCH, **kw2}
    return L.flint_qk_norm_rope_paged_kv(qkv, b["T"], b["hq"], b["hkv"], b["dh"], qw, kw, cs, max_pos, rope, eps,
                                         b["qs"], b["kl"], b["B"], b["bt"], b["mp"], b["page"], b["pages"], b["dt"],
                                         b["ks"], b["vs"], q_out, b["k"], b["v"], None, None)


def _attn(L, q=A, out=A, max_q=1, window=0, scale=0.088, ws=A, ws_bytes=1 << 40, **kw2):
    b = {**BATCH, **kw2}
    return L.flint_paged_attention(q, b["T"], b["qs"], b["kl"], b["B"], b["bt"], b["mp"], b["page"], b["pages"],
                                   b["k"], b["v"], b["dt"], b["ks"], b["vs"], b["hq"], b["hkv"], b["dh"], max_q,
                                   window, scale, out, ws, ws_bytes, None, None)


@pytest.mark.parametrize("bad,rc", BAD_BATCH)
def test_batch_arguments(L, bad, rc):
    assert _append(L, **bad) == rc
    assert _attn(L, **bad) == rc
    assert fm.flint_last_error()


def test_append_arguments(L):
    assert _append(L, qkv=None) == -1
    assert _append(L, q_out=None) == -1
    assert _append(L, qw=None) == -1          # one weight without the other
    assert _append(L, cs=None) == -1
    assert _append(L, max_pos=0) == -1
    assert _append(L, eps=-1.0) == -1
    assert _append(L, eps=float("nan")) == -1
    assert _append(L, qkv=A + 8) == -3
    assert _append(L, cs=A + 4) == -3
    assert _append(L, T=0) == 0
    assert _append(L, B=0) == 0


def test_attention_arguments(L):
    assert _attn(L, q=None) == -1
    assert _attn(L, out=None) == -1
    assert _attn(L, q=A + 8) == -3
    assert _attn(L, ws=A + 8) == -3
    assert _attn(L, hq=34, hkv=2) == -2       # 17 query heads per kv head
    assert _attn(L, hq=30) == -2
    assert _attn(L, hq=2048, hkv=128) == -2
    assert _attn(L, B=32769) == -2
    assert _attn(L, max_q=0) == -1
    assert _attn(L, pages=0) == -1
    assert _attn(L, window=-1) == -1
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(L, scale=s) == -1
    assert _attn(L, T=0) == 0
    assert _attn(L, B=0) == 0
    for mq in (1, 2, 3, 100):
        need = fm.flint_paged_attention_workspace_bytes(4, 2, 32, 4, mq)
        assert need > 0
        assert _attn(L, max_q=mq, ws_bytes=need - 1) == -4
        assert _attn(L, max_q=mq, ws=None) == -4
    for bad in ((0, 2, 32, 4, 1), (4, 0, 32, 4, 1), (4, 2, 30, 4, 1), (4, 2, 34, 2, 1), (4, 2, 32, 4, 0)):
        assert fm.flint_paged_attention_workspace_bytes(*bad) == 0


def _sample(L, logits=A, rows=2, vocab=100, stride=100, dt=0, t=A, k=A, p=A, m=A, u=A, tok=A, lp=A):
    return L.flint_sample(logits, rows, vocab, stride, dt, t, k, p, m, u, tok, lp, None, None)


def test_sample_arguments(L):
    assert _sample(L, dt=2) == -1
    assert _sample(L, rows=-1) == -1
    assert _sample(L, vocab=0) == -1
    assert _sample(L, stride=99) == -1
    assert _sample(L, vocab=(1 << 24) + 1, stride=1 << 25) == -2
    for name in ("logits", "u", "tok"):
        assert _sample(L, **{name: None}) == -1
    for name in ("logits", "t", "k", "p", "m", "u", "tok", "lp"):
        assert _sample(L, **{name: A + 2}) == -3
    assert _sample(L, logits=A + 1, dt=1) == -3
    assert _sample(L, rows=0) == 0


def test_python_wrappers_refuse_cpu_tensors():
    import torch
    x = torch.zeros(1000)
    with pytest.raises(fm.FlintError) as e:
        fm.flint_sample(x, 1, 100, 100, fm.FLINT_LOGITS_F32, None, None, None, None, x, x)
    assert e.value.code == -1 and "logits" in str(e.value)
    with pytest.raises(fm.FlintError):  # torch's own exceptions do not leave the marshalling
        fm.flint_sample(x.to_sparse(), 1, 100, 100, fm.FLINT_LOGITS_F32, None, None, None, None, x, x)
    with pytest.raises(fm.FlintError):
        fm.flint_sample(A, 1 << 40, 100, 100, fm.FLINT_LOGITS_F32, None, None, None, None, A, A, stream=0)
    with pytest.raises(fm.FlintError):
        fm.flint_qk_norm_rope_paged_kv(x, 1, 1, 1, None, None, None, 0, False, 0.0, x, x, 1, x, 1, 16, 4,
                                       fm.FLINT_KV_BF16, None, None, x, x, x)
    with pytest.raises(fm.FlintError):
        fm.flint_paged_attention(x, 1, x, x, 1, x, 1, 16, 4, x, x, fm.FLINT_KV_BF16, None, None, 1, 1, 1, 0, 0.1, x, x)
    with pytest.raises(TypeError):
        fm.flint_sample("logits", 1, "many", 100, 0, None, None, None, None, x, x)


@pytest.mark.parametrize("rows,stride", [(3, 1 << 62), (2, (1 << 63) - 1), ((1 << 24), 1 << 40), (2, 901)])
def test_sample_refuses_strides_past_the_tensor(rows, stride):
    # the bytes that rows * row_stride reach, where they do not fit 64 bits either
    import torch
    x, per_row = torch.zeros(1000), torch.zeros(1 << 24)
    with pytest.raises(fm.FlintError) as e:
        fm.flint_sample(x, rows, 100, stride, fm.FLINT_LOGITS_F32, None, None, None, None, per_row, per_row)
    assert e.value.code == -1 and "logits" in str(e.value) and "needed" in str(e.value)


@pytest.mark.parametrize("by", [1, 2, 3])
def test_misaligned_status(L, by):
    # the kernels set it with a 32-bit atomic
    assert L.flint_qk_norm_rope_paged_kv(A, 4, 32, 4, 128, A, A, A, 16, 1, 1e-6, A, A, 2, A, 8, 16, 64, 0, None, None, A,
                                         A, A, A + by, None) == -3
    assert L.flint_paged_attention(A, 4, A, A, 2, A, 8, 16, 64, A, A, 0, None, None, 32, 4, 128, 1, 0, 0.088, A, A,
                                   1 << 40, A + by, None) == -3
    assert L.flint_sample(A, 2, 100, 100, 0, A, A, A, A, A, A, A, A + by, None) == -3


def _sample_tensors():
    import torch
    i32, f32 = torch.int32, torch.float32
    return dict(logits=torch.zeros((4, 200)), rows=4, vocab=200, row_stride=200, logits_dtype=fm.FLINT_LOGITS_F32,
                temperature=torch.zeros(4, dtype=f32), top_k=torch.zeros(4, dtype=i32), top_p=torch.zeros(4, dtype=f32),
                min_p=torch.zeros(4, dtype=f32), u=torch.zeros(4, dtype=f32), tokens=torch.zeros(4, dtype=i32),
                logprobs=torch.zeros(4, dtype=f32), status=torch.zeros(1, dtype=i32))


def _paged_tensors(e4m3, attention):
    import torch
    i32, bf16 = torch.int32, torch.bfloat16
    pool = lambda: torch.zeros((4, 16, 2, 128), dtype=torch.float8_e4m3fn if e4m3 else bf16)  # noqa: E731
    d = dict(T=3, q_start=torch.zeros(3, dtype=i32), kv_len=torch.zeros(2, dtype=i32), B=2,
             block_table=torch.zeros((2, 5), dtype=i32), max_pages=5, page_size=16, n_pages=4, k_cache=pool(),
             v_cache=pool(), cache_dtype=fm.FLINT_KV_E4M3 if e4m3 else fm.FLINT_KV_BF16,
             k_scale=torch.ones(2) if e4m3 else None, v_scale=torch.ones(2) if e4m3 else None, n_q_heads=4,
             n_kv_heads=2, status=torch.zeros(1, dtype=i32))
    q = lambda h: torch.zeros((3, h, 128), dtype=bf16)  # noqa: E731
    if attention:
        return dict(d, q=q(4), max_q_len=1, window=0, scale=0.1, out=q(4), workspace=torch.zeros(64, dtype=torch.uint8))
    w = lambda: torch.ones(128, dtype=bf16)  # noqa: E731
    return dict(d, qkv=q(8), q_norm_w=w(), k_norm_w=w(), cos_sin=torch.zeros((9, 128)), max_pos=9, rope=True, eps=0.0,
                q_out=q(4))


def _calls():
    return [(fm.flint_sample, _sample_tensors()),
            *[(f, _paged_tensors(e, f is fm.flint_paged_attention))
              for f in (fm.flint_paged_attention, fm.flint_qk_norm_rope_paged_kv) for e in (False, True)]]


def test_element_types():
    """Each tensor of another type than the kernel reads is refused by name, wider ones (torch's default integers) too;
    the right type gets as far as the device check. Every other tensor is an address here, so that the one under test is
    the first to be looked at."""
    import torch
    for f, args in _calls():
        for name, x in args.items():
            if not isinstance(x, torch.Tensor):
                continue
            only = {k: A if isinstance(v, torch.Tensor) else v for k, v in args.items()}
            with pytest.raises(fm.FlintError) as e:  # the right type: refused for its device only
                f(**{**only, name: x}, stream=0)
            assert name in str(e.value) and "CUDA tensor" in str(e.value)
            if name == "workspace":
                continue
            for dt in (torch.int64, torch.float64, torch.float32, torch.int32, torch.float16, torch.bfloat16, torch.bool,
                       torch.float8_e5m2):
                if dt == x.dtype:
                    continue
                with pytest.raises(fm.FlintError) as e:
                    f(**{**only, name: torch.zeros((x.numel() * 2,), dtype=dt)}, stream=0)
                assert e.value.code == -1 and name in str(e.value) and "element type" in str(e.value), (name, dt)
            with pytest.raises(fm.FlintError) as e:
                f(**{**only, name: True}, stream=0)
            assert name in str(e.value)


def test_bits_of_16_and_8_bit_types():
    import torch
    for f, args in _calls()[1:]:
        for name in ("q", "qkv", "q_norm_w", "out", "q_out", "k_cache", "v_cache"):
            if name not in args:
                continue
            only = {k: A if isinstance(v, torch.Tensor) else v for k, v in args.items()}
            one = args[name].element_size() == 1
            for dt in (torch.uint8, torch.int8) if one else (torch.int16, torch.uint16):
                with pytest.raises(fm.FlintError) as e:
                    f(**{**only, name: args[name].view(dt)}, stream=0)
                assert name in str(e.value) and "CUDA tensor" in str(e.value)


def test_workspace_is_a_tensor():
    # an address has no size: refused as such, not as too small
    for e4m3 in (False, True):
        import torch
        args = {k: A if isinstance(v, torch.Tensor) else v for k, v in _paged_tensors(e4m3, True).items()}
        with pytest.raises(fm.FlintError) as e:
            fm.flint_paged_attention(**args, stream=0)
        assert e.value.code == -1 and "workspace" in str(e.value) and "tensor" in str(e.value)


def test_attention_workspace_is_bounded(L):
    # partials are kept only where a kv head's work is cut: 39 MB at most for prompt pieces, 5 MB and the prefix sums for
    # decode steps, whatever the number of kv heads
    for hkv in list(range(1, 160)) + [296, 297, 512, 1024]:
        assert 0 < fm.flint_paged_attention_workspace_bytes(4096, 1, hkv, hkv, 4096) < 39.5e6, hkv
        assert 0 < fm.flint_paged_attention_workspace_bytes(64, 64, hkv, hkv, 1) < 5.2e6, hkv
    assert fm.flint_paged_attention_workspace_bytes(4096, 1, 1024, 1024, 4096) < 1e5


def test_attention_workspace_serves_smaller_calls(L):
    # sized once for the largest step, as the README has it
    sizes = ((1, 1, 1), (2, 1, 2), (16, 4, 16), (64, 64, 1), (64, 5, 17), (300, 64, 200), (4096, 3000, 1),
             (4096, 32768, 4096), (1 << 24, 32768, 1 << 24))
    for hkv in (1, 4, 37, 74, 75, 100, 148, 149, 297, 1024):
        for group in (1, 8):
            if hkv * group > 1024:
                continue
            need = {x: fm.flint_paged_attention_workspace_bytes(x[0], x[1], hkv * group, hkv, x[2]) for x in sizes}
            for x, nx in need.items():
                for y, ny in need.items():
                    if all(a <= b for a, b in zip(x, y)):
                        assert nx <= ny, (hkv, group, x, y)
