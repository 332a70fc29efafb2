"""Host-side validation of the attention step's entry points; no GPU is needed.

The cases pass arguments that the host checks must reject before any launch,
and run only where no GPU device node exists (tests/test_abi.py).  They run
once more against a build of the library whose host code carries the address
and undefined-behaviour sanitizers.
"""

import ctypes
import importlib.util
import os
import shutil
import subprocess
import sys
from ctypes import c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NO_GPU = not os.path.exists("/dev/kfd")
SANITIZED_LIB = os.environ.get("ENGRAM_ABI_SANITIZED_LIB")
OK, ARG, UNSUPPORTED = 0, 1, 2
BF16, MXFP8 = 0, 1
FAKE = 0x10000      # aligned, never dereferenced by the host checks


class Cache(ctypes.Structure):
    _fields_ = [("fmt", c_int), ("pages", c_int32), ("kv_heads", c_int32), ("page_size", c_int32),
                ("head_dim", c_int32), ("k", c_void_p), ("v", c_void_p), ("k_scales", c_void_p),
                ("v_scales", c_void_p)]


def cache(**kw):
    a = dict(fmt=BF16, pages=4, kv_heads=2, page_size=16, head_dim=128, k=FAKE, v=FAKE,
             k_scales=None, v_scales=None)
    a.update(kw)
    return Cache(*a.values())


@pytest.fixture(scope="module")
def lib():
    path = SANITIZED_LIB
    if not path:
        import __graft_entry__
        __graft_entry__._ensure_built()
        path = os.path.join(ROOT, "gram_hash_memory_amd", "libengram.so")
    lib = ctypes.CDLL(path)
    lib.engram_last_error.restype = ctypes.c_char_p
    P = c_void_p
    lib.engram_cache_write.argtypes = [P, P, c_int64, c_int64, P, c_int64, c_int64, P, c_int32, P, P]
    lib.engram_cache_read.argtypes = [P, P, c_int32, P, P, P, P]
    lib.engram_qk_norm_rope.argtypes = [P, c_int64] + [c_int32] * 4 + [P, P, c_float, P, P, c_int32,
                                                                       c_int32] + [P] * 6
    lib.engram_paged_attention_workspace_bytes.argtypes = [c_int32] * 5
    lib.engram_paged_attention_workspace_bytes.restype = c_size_t
    lib.engram_paged_attention.argtypes = [P, P, P, c_int32, P, c_int32, c_int32, c_int32, c_float,
                                           c_int32, P, P, P, c_size_t, P, P]
    lib.engram_quantize_mxfp4.argtypes = [P, c_int32, c_int32, P, P, P]
    lib.engram_project_mxfp4.argtypes = [P] * 4 + [c_int32] * 3 + [P]
    return lib


def caller(fn, order, ok):
    """fn with the arguments ok, some replaced; the cache a struct or None."""
    def call(**kw):
        a = dict(ok, **kw)
        c = a.get("cache")
        if isinstance(c, Cache):
            a["cache"] = ctypes.byref(c)
        return fn(*[a[n] for n in order])
    return call


BAD_CACHES = [(None, ARG), (cache(fmt=7), ARG), (cache(pages=0), ARG), (cache(kv_heads=0), ARG),
              (cache(page_size=12), UNSUPPORTED), (cache(page_size=4), UNSUPPORTED),
              (cache(page_size=8192), UNSUPPORTED), (cache(page_size=0), UNSUPPORTED),
              (cache(page_size=-16), UNSUPPORTED), (cache(head_dim=48), UNSUPPORTED),
              (cache(head_dim=288), UNSUPPORTED), (cache(head_dim=0), UNSUPPORTED),
              (cache(k=None), ARG), (cache(v=FAKE + 8), ARG), (cache(fmt=MXFP8), ARG),
              (cache(fmt=MXFP8, k_scales=FAKE), ARG),
              (cache(fmt=MXFP8, k_scales=FAKE, v_scales=FAKE + 4), ARG),
              (cache(k_scales=FAKE, v_scales=FAKE), ARG)]


@pytest.mark.skipif(not NO_GPU, reason="validation-rejection cases run only without a GPU")
class TestValidation:
    def test_cache_write_rejects(self, lib):
        call = caller(lib.engram_cache_write,
                      ("cache", "k", "kt", "kh", "v", "vt", "vh", "slots", "T", "bad", "stream"),
                      dict(cache=cache(), k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, slots=FAKE,
                           T=3, bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw in (dict(T=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2),
                   dict(kt=-8), dict(vt=12), dict(kh=120), dict(vh=129), dict(vh=132),
                   dict(slots=None), dict(slots=FAKE + 4), dict(bad=FAKE + 2)):
            assert call(**kw) == ARG, kw
        assert call(T=0, k=None, v=None, slots=None) == OK
        big = cache(kv_heads=1 << 20)
        assert call(cache=big, T=1 << 20) == UNSUPPORTED
        assert b"too many" in lib.engram_last_error()

    def test_cache_read_rejects(self, lib):
        call = caller(lib.engram_cache_read, ("cache", "slots", "T", "k", "v", "bad", "stream"),
                      dict(cache=cache(), slots=FAKE, T=3, k=FAKE, v=FAKE, bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw in (dict(T=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2),
                   dict(slots=None), dict(slots=FAKE + 4), dict(bad=FAKE + 2)):
            assert call(**kw) == ARG, kw
        assert call(T=0, k=None, v=None, slots=None) == OK
        assert call(cache=cache(kv_heads=1 << 20), T=1 << 20) == UNSUPPORTED

    def test_qk_norm_rope_rejects(self, lib):
        call = caller(lib.engram_qk_norm_rope,
                      ("qkv", "stride", "T", "hq", "hkv", "D", "qw", "kw", "eps", "pos", "inv", "rot",
                       "inter", "q", "k", "cache", "slots", "bad", "stream"),
                      dict(qkv=FAKE, stride=1024, T=3, hq=4, hkv=2, D=128, qw=FAKE, kw=FAKE, eps=1e-6,
                           pos=FAKE, inv=FAKE, rot=64, inter=0, q=FAKE, k=FAKE, cache=None, slots=None,
                           bad=None, stream=None))
        for kw in (dict(T=-1), dict(hq=0), dict(hkv=0), dict(hkv=-2), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(stride=760), dict(stride=1028), dict(qkv=None),
                   dict(qkv=FAKE + 8), dict(q=None), dict(q=FAKE + 4), dict(k=FAKE + 4), dict(k=None),
                   dict(qw=None), dict(kw=FAKE + 2), dict(pos=None), dict(pos=FAKE + 2),
                   dict(inv=None), dict(inv=FAKE + 4), dict(slots=FAKE), dict(bad=FAKE)):
            assert call(**kw) == ARG, kw
        for kw in (dict(D=40), dict(D=512), dict(rot=0), dict(rot=-16), dict(rot=24), dict(rot=144),
                   dict(hq=1 << 30)):
            assert call(**kw) == UNSUPPORTED, kw
        with_cache = dict(cache=cache(), slots=FAKE, k=None)
        for c, status in BAD_CACHES[1:]:
            assert call(**dict(with_cache, cache=c)) == status
        for kw in (dict(slots=None), dict(slots=FAKE + 4), dict(bad=FAKE + 1), dict(stride=1016),
                   dict(cache=cache(kv_heads=4)), dict(cache=cache(head_dim=64))):
            assert call(**dict(with_cache, **kw)) == ARG, kw
        assert call(T=0, qkv=None, q=None) == OK
        assert call(T=0, stride=8) == ARG
        assert call(T=(1 << 31) - 1, hq=1 << 12, stride=1 << 20) == UNSUPPORTED

    def test_paged_attention_rejects(self, lib):
        need = lib.engram_paged_attention_workspace_bytes(2, 8, 2, 128, 100000)
        call = caller(lib.engram_paged_attention,
                      ("cache", "q", "table", "width", "lens", "n", "hq", "max_len", "scale", "window",
                       "out", "lse", "ws", "ws_bytes", "bad", "stream"),
                      dict(cache=cache(), q=FAKE, table=FAKE, width=4, lens=FAKE, n=2, hq=8,
                           max_len=100000, scale=0.1, window=0, out=FAKE, lse=None, ws=FAKE,
                           ws_bytes=need, bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw in (dict(n=-1), dict(max_len=-1), dict(window=-1), dict(width=-1), dict(hq=0), dict(hq=7),
                   dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(q=FAKE + 8),
                   dict(out=None), dict(out=FAKE + 8), dict(lens=None), dict(lens=FAKE + 2),
                   dict(table=None), dict(table=FAKE + 1), dict(lse=FAKE + 2), dict(bad=FAKE + 2)):
            assert call(**kw) == ARG, kw
        assert call(n=0, q=None, out=None, lens=None, table=None) == OK
        assert call(n=(1 << 31) - 1, max_len=0) == UNSUPPORTED

    def test_paged_attention_rejects_a_short_workspace(self, lib):
        need = lib.engram_paged_attention_workspace_bytes(1, 8, 2, 128, 100000)
        if need == 0:
            pytest.skip("no sequence is split")
        call = lambda ws, nbytes: lib.engram_paged_attention(  # noqa: E731
            ctypes.byref(cache()), FAKE, FAKE, 4, FAKE, 1, 8, 100000, 0.1, 0, FAKE, None, ws, nbytes,
            None, None)
        assert call(None, need) == ARG and call(FAKE + 16, need) == ARG and call(FAKE, need - 1) == ARG

    def test_workspace_bytes_of_nonsense_is_zero(self, lib):
        f = lib.engram_paged_attention_workspace_bytes
        for a in ((0, 8, 2, 128, 9), (-1, 8, 2, 128, 9), (1, 7, 2, 128, 9), (1, 8, 0, 128, 9),
                  (1, 8, 2, 100, 9), (1, 8, 2, 128, 0), (1, 8, 2, 128, -5)):
            assert f(*a) == 0, a

    def test_workspace_never_shrinks_with_length(self, lib):
        """A window or shorter lengths need no more than max_len asked for."""
        f = lib.engram_paged_attention_workspace_bytes
        for n, hq, hkv in ((1, 32, 8), (3, 6, 2), (64, 32, 8), (700, 8, 8), (2, 128, 1)):
            sizes = [f(n, hq, hkv, 128, length) for length in
                     (1, 7, 31, 32, 33, 100, 500, 1000, 4096, 4097, 50000, 131072, 1 << 20, (1 << 31) - 1)]
            assert sizes == sorted(sizes), (n, hq, hkv)

    def test_paged_attention_rejects_lengths_past_32_bits_of_places(self, lib):
        c = cache()
        call = lambda max_len, n=1: lib.engram_paged_attention(  # noqa: E731
            ctypes.byref(c), FAKE, FAKE, 4, FAKE, n, 8, max_len, 1.0, 0, FAKE, None, FAKE, 1 << 40, None, None)
        assert call((1 << 30) + 1) == UNSUPPORTED
        assert call(1 << 30, n=1 << 20) == UNSUPPORTED

    def test_fp4_rejects(self, lib):
        call = caller(lib.engram_quantize_mxfp4, ("w", "N", "K", "codes", "scales", "stream"),
                      dict(w=FAKE, N=8, K=64, codes=FAKE, scales=FAKE, stream=None))
        for kw in (dict(N=-1), dict(K=0), dict(K=48), dict(w=None), dict(w=FAKE + 8), dict(codes=None),
                   dict(codes=FAKE + 8), dict(scales=None)):
            assert call(**kw) == ARG, kw
        assert call(N=0, w=None) == OK
        call = caller(lib.engram_project_mxfp4, ("x", "codes", "scales", "out", "T", "K", "N", "stream"),
                      dict(x=FAKE, codes=FAKE, scales=FAKE, out=FAKE, T=3, K=64, N=5, stream=None))
        for kw in (dict(T=-1), dict(K=0), dict(K=33), dict(N=0), dict(x=None), dict(x=FAKE + 8),
                   dict(codes=None), dict(codes=FAKE + 8), dict(scales=None), dict(out=None),
                   dict(out=FAKE + 2)):
            assert call(**kw) == ARG, kw
        assert call(T=0, x=None, out=None) == OK
        assert call(K=1 << 20, N=1 << 20) == UNSUPPORTED
        assert call(K=1 << 20, T=1 << 20, N=1) == UNSUPPORTED

    def test_fp4_rejects_more_tiles_than_a_grid_holds(self, lib):
        call = lambda T, N: lib.engram_project_mxfp4(FAKE, FAKE, FAKE, None, T, 32, N, None)  # noqa: E731
        assert call(1 << 24, 1 << 20) == UNSUPPORTED
        assert call(128, 1 << 20) == ARG                    # not too many: the missing output is what it minds


class TestBinding:
    """What the Python binding refuses before it reaches the library (no GPU tensors needed)."""

    def test_cache_wants_gpu_tensors_and_scales_that_fit(self):
        if SANITIZED_LIB:
            pytest.skip("the binding needs torch")
        import torch
        import gram_hash_memory_amd as eg
        k = torch.zeros(2, 1, 8, 32, dtype=torch.int16)
        with pytest.raises(TypeError, match="GPU"):
            eg.KVCache(eg.ENGRAM_CACHE_BF16, k, k)
        with pytest.raises(ValueError, match="scales"):
            eg.KVCache(eg.ENGRAM_CACHE_MXFP8, k, k)
        with pytest.raises(ValueError, match="scales"):
            eg.KVCache(eg.ENGRAM_CACHE_BF16, k, k, k, k)
        with pytest.raises(ValueError, match="must both"):
            eg.KVCache(eg.ENGRAM_CACHE_BF16, k, k[:1])
        with pytest.raises(ValueError, match="unknown"):
            eg.KVCache(9, k, k)


@pytest.mark.skipif(not NO_GPU, reason="the rejection cases run only without a GPU")
@pytest.mark.skipif(bool(SANITIZED_LIB), reason="already inside the sanitized run")
@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs hipcc")
def test_validation_under_address_and_ub_sanitizers():
    spec = importlib.util.spec_from_file_location(
        "_engram_build_sanitized2", os.path.join(ROOT, "gram_hash_memory_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    lib = b.SANITIZED_LIB
    mark = b"engram-build-id " + b.build_id().encode() + b"\0"
    if not (os.path.exists(lib) and mark in open(lib, "rb").read()):
        lib = b.build_sanitized()
    env = dict(os.environ, LD_PRELOAD=b.sanitizer_runtime(), ENGRAM_ABI_SANITIZED_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=24")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.abspath(__file__), "-k", "TestValidation"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
