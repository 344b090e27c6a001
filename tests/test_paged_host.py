"""Host-side checks of the paged-cache entry points (no GPU needed): every bad
argument is refused with its documented status before CUDA is touched, and the
binding raises on tensors it cannot pass on."""
import pytest
import torch

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3

# Fake device addresses: never dereferenced, every call below fails (or ends
# in) a host check.
A = 0x7F0000000000


def cache(lib, **kw):
    from gated_deltanet_chunkwise_gb300 import abi
    f = dict(ck=A, cv=A + 0x1000, kp=4096, kh=2048, kt=128, vp=4096, vh=2048,
             vt=128, table=A + 0x2000, ts=4, lens=A + 0x3000, pages=8, page=16,
             width=4, heads=2, d=128, dtype=0)
    f.update(kw)
    return abi._PAGED_CACHE.pack(*f.values())


def append(lib, q=A, qs=512, k=A + 0x4000, ks=256, v=A + 0x5000, vs=256,
           qo=A + 0x6000, qos=512, rope=A + 0x7000, rows=64, rot=128, pos=None,
           axes=1, sections=None, inter=0, cu=None, B=1, T=1, Hq=4, **kw):
    import ctypes
    sec = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    return lib.library().gdn_paged_append(
        q, qs, k, ks, v, vs, qo, qos, rope, rows, rot, pos, axes, sec, inter,
        cache(lib, **kw), cu, B, T, Hq, None)


def attn(lib, q=A, qs=512, cu=None, B=1, T=1, Hq=4, scale=0.1, causal=1,
         window=0, out=A + 0x8000, lse=None, path=0, **kw):
    return lib.library().gdn_paged_attn(q, qs, cache(lib, **kw), cu, B, T, Hq,
                                        scale, causal, window, out, lse, path,
                                        None)


CACHE = [
    (dict(ck=0), INVALID), (dict(cv=0), INVALID),
    (dict(table=0), INVALID), (dict(lens=0), INVALID),
    (dict(pages=0), INVALID), (dict(width=0), INVALID),
    (dict(heads=0), INVALID), (dict(ts=3), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=512), UNSUPPORTED), (dict(width=1 << 27, ts=1 << 27), UNSUPPORTED),
    (dict(kp=4), INVALID), (dict(vh=-8), INVALID), (dict(kt=64), INVALID),
    (dict(vt=120), INVALID), (dict(kp=1 << 40), INVALID),
    (dict(kh=0), INVALID), (dict(vh=64), INVALID), (dict(vp=0), INVALID),
    (dict(ck=A + 8), MISALIGNED), (dict(cv=A + 2), MISALIGNED),
    (dict(table=A + 2), MISALIGNED), (dict(lens=A + 1), MISALIGNED),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(cu=A, B=0), INVALID), (dict(cu=A + 2), MISALIGNED),
    (dict(B=1 << 16, T=1 << 16), UNSUPPORTED),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(cu=A, T=(1 << 30) + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", CACHE)
def test_cache_and_batch_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect
    assert attn(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(qo=None), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(rot=8), UNSUPPORTED),
    (dict(rope=None), INVALID), (dict(rows=0), INVALID),
    (dict(rot=0, pos=A), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(axes=2, sections=[32, 32]), INVALID),          # no positions
    (dict(axes=2, pos=A), INVALID),                      # no sections
    (dict(axes=2, pos=A, sections=[32, 31]), INVALID),
    (dict(axes=2, pos=A, sections=[-1, 65]), INVALID),
    (dict(axes=3, pos=A, sections=[64, 64, 64]), INVALID),
    (dict(qs=504), INVALID), (dict(ks=260), INVALID), (dict(vs=128), INVALID),
    (dict(qos=0), INVALID), (dict(qo=A, qos=1024), INVALID),
    (dict(q=A + 4), MISALIGNED), (dict(rope=A + 4), MISALIGNED),
    (dict(pos=A + 2), MISALIGNED),
    (dict(T=0), OK), (dict(B=0), OK), (dict(T=0, ck=0), INVALID),
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=A), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(path=3), INVALID), (dict(path=-1), INVALID),
    (dict(Hq=3), INVALID), (dict(Hq=260, qs=260 * 128), UNSUPPORTED),
    (dict(qs=256), INVALID), (dict(qs=516), INVALID),
    (dict(q=A + 4), MISALIGNED), (dict(out=A + 8), MISALIGNED),
    (dict(lse=A + 2), MISALIGNED), (dict(T=0), OK), (dict(B=0), OK),
])
def test_attn_refusals(lib, kw, expect):
    assert attn(lib, **kw) == expect


def tensors(dtype=torch.bfloat16):
    kc = torch.zeros(4, 2, 16, 128, dtype=dtype)
    return dict(q=torch.zeros(2, 3, 4, 128, dtype=dtype),
                k=torch.zeros(2, 3, 2, 128, dtype=dtype),
                v=torch.zeros(2, 3, 2, 128, dtype=dtype), k_cache=kc,
                v_cache=kc.clone(), page_table=torch.zeros(2, 2, dtype=torch.int32),
                kv_lens=torch.full((2,), 5, dtype=torch.int32))


def test_binding_refuses_cpu_tensors(lib):
    t = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        lib.gdn_paged_append(**t)
    del t["k"], t["v"]
    with pytest.raises(ValueError, match="CUDA"):
        lib.gdn_paged_attn(**t)


def test_packed_struct_matches_the_header(lib):
    """The packed cache has the C struct's layout (natural alignment)."""
    import ctypes

    from gated_deltanet_chunkwise_gb300 import abi

    class C(ctypes.Structure):
        _fields_ = ([("p%d" % i, ctypes.c_void_p) for i in range(2)]
                    + [("s%d" % i, ctypes.c_int64) for i in range(6)]
                    + [("table", ctypes.c_void_p), ("ts", ctypes.c_int64),
                       ("lens", ctypes.c_void_p)]
                    + [("i%d" % i, ctypes.c_int) for i in range(6)])
    raw = abi._PAGED_CACHE.pack(*range(1, 18))
    assert len(raw) == ctypes.sizeof(C)
    c = C.from_buffer_copy(raw)
    assert [getattr(c, f[0]) for f in C._fields_] == list(range(1, 18))


def test_a_failed_mark_leaves_the_stream_as_it_was(lib, monkeypatch):
    """An input that cannot be marked as used on the given stream: the error
    comes out and no stream context stays entered."""
    from gated_deltanet_chunkwise_gb300 import abi
    depth = []

    class Context:
        def __init__(self, *args):
            pass

        def __enter__(self):
            depth.append(1)

        def __exit__(self, *args):
            depth.pop()

    class Bad:
        def record_stream(self, stream):
            raise RuntimeError("no")

    class Stream:
        cuda_stream = 7

    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch.cuda, "device", Context)
    with pytest.raises(RuntimeError, match="no"):
        abi._paged_stream(Stream(), torch.device("cuda:0"), (None, Bad()))
    assert not depth
    raw, ctx = abi._paged_stream(Stream(), torch.device("cuda:0"), (None,))
    assert raw == 7 and depth == [1]
    ctx.__exit__(None, None, None)
    assert not depth


def test_empty_batch(lib):
    """A batch of no sequences has empty tensors, whose addresses are null."""
    none = dict(B=0, table=0, lens=0, ts=4)
    assert attn(lib, q=None, out=None, **none) == OK
    assert append(lib, q=None, k=None, v=None, qo=None, **none) == OK
    assert attn(lib, **dict(none, B=1)) == INVALID
    assert append(lib, **dict(none, B=1)) == INVALID


@pytest.mark.parametrize("kw,expect", [
    # 5 tokens of 4 heads of 128: 5120 bytes each, one after the other or apart
    (dict(T=5, out=A + 16), INVALID), (dict(T=5, out=A - 16), INVALID),
    (dict(T=5, out=A + 5104), INVALID), (dict(T=5, out=A - 5104), INVALID),
    (dict(T=5, qs=1024, out=A + 9200), INVALID),
    (dict(T=0, out=A), OK),
])
def test_output_over_the_queries(lib, kw, expect):
    """An output that lies over part of the queries would be written while other
    blocks still read them."""
    assert attn(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    # fused rows of 8 heads of 128: 4 of queries, 2 of keys, 2 of values
    (dict(qo=A + 2 * 512), INVALID),                  # over the keys
    (dict(qo=A + 2 * 128), INVALID),                  # half over the queries
    (dict(qo=A - 2 * 128), INVALID),                  # and over the last values
    (dict(qo=A + 2 * 1024), INVALID),                 # a row further
    (dict(qo=A, qos=512), INVALID), (dict(qo=A + 64, qos=512), INVALID),
    (dict(T=0, qo=A + 2 * 128), OK),
])
def test_append_output_over_the_inputs(lib, kw, expect):
    f = dict(T=5, q=A, qs=1024, k=A + 2 * 512, ks=1024, v=A + 2 * 768, vs=1024,
             qos=1024)
    assert append(lib, **dict(f, **kw)) == expect
    # in place, or beside them: past the checks (and no further without a GPU)
    for qo, qos in ((A, 1024), (A + (1 << 20), 512)):
        if not torch.cuda.is_available():
            assert append(lib, **dict(f, qo=qo, qos=qos)) not in (INVALID, UNSUPPORTED)
