"""Host-side validation of the attention of chunks and shared prefixes, of places' weights and of eviction; no GPU.

As tests/test_abi_attention.py: the cases pass arguments that the host checks must reject before any launch, run only
where no GPU device node exists, and run once more under the address and undefined-behaviour sanitizers.
"""

import ctypes
import os
import subprocess
import sys
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p

import pytest

import test_abi_attention as base
from test_abi_attention import ARG, BAD_CACHES, FAKE, NO_GPU, OK, UNSUPPORTED, cache, caller

INF, NAN = float("inf"), float("nan")


class Rules(ctypes.Structure):
    _fields_ = [("window", c_int32), ("cap", c_float), ("slopes", c_void_p), ("doc_starts", c_void_p),
                ("prefix_lens", c_void_p)]


@pytest.fixture(scope="module")
def lib():
    path = base.SANITIZED_LIB
    if not path:
        import __graft_entry__
        __graft_entry__._ensure_built()
        path = os.path.join(base.ROOT, "gram_hash_memory_amd", "libengram.so")
    lib = ctypes.CDLL(path)
    lib.engram_last_error.restype = ctypes.c_char_p
    P, i, n = c_void_p, c_int32, c_size_t
    lib.engram_chunk_attention_workspace_bytes.argtypes = [i] * 6
    lib.engram_chunk_attention_workspace_bytes.restype = n
    lib.engram_chunk_attention.argtypes = [P, P, i, P, P, i, P, i, i, i, P, c_float, P, P, P, n, P, P]
    lib.engram_shared_prefix_attention_workspace_bytes.argtypes = [i] * 7
    lib.engram_shared_prefix_attention_workspace_bytes.restype = n
    lib.engram_shared_prefix_attention.argtypes = [P, P, P, P, i, P, i, i, P, i, P, i, i, i, c_float, P, P, P, n, P, P]
    lib.engram_cache_weights.argtypes = [P, P, i, P, P, i, P, i, i, i, P, c_float, P, P, c_int64, P, P]
    lib.engram_cache_evict.argtypes = [P, P, i, P, i, i, i, i, i, P, c_int64, P, i, P, P, c_int64, P, P, P]
    return lib


def rules(**kw):
    return ctypes.pointer(Rules(**kw))


BAD_RULES = [dict(window=-1), dict(cap=-1.0), dict(cap=NAN), dict(cap=INF), dict(slopes=FAKE + 2), dict(doc_starts=FAKE + 1),
             dict(prefix_lens=FAKE + 3)]
SEQUENCES = [(dict(n=-1), ARG), (dict(max_len=-1), ARG), (dict(max_len=(1 << 30) + 1), UNSUPPORTED), (dict(width=-1), ARG),
             (dict(heads=0), ARG), (dict(heads=-2), ARG), (dict(heads=3), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG),
             (dict(lens=None), ARG), (dict(lens=FAKE + 2), ARG), (dict(table=None), ARG), (dict(table=FAKE + 1), ARG),
             (dict(bad=FAKE + 2), ARG), (dict(q=None), ARG), (dict(q=FAKE + 8), ARG), (dict(lse=FAKE + 2), ARG)]


@pytest.mark.skipif(not NO_GPU, reason="validation-rejection cases run only without a GPU")
class TestValidation:
    def test_chunk_attention_rejects(self, lib):
        need = lib.engram_chunk_attention_workspace_bytes(10, 3, 8, 2, 128, 100)
        assert need > 0
        call = caller(lib.engram_chunk_attention,
                      ("cache", "q", "T", "cu", "table", "width", "lens", "n", "heads", "max_len", "rules", "scale", "out",
                       "lse", "ws", "bytes", "bad", "stream"),
                      dict(cache=cache(), q=FAKE, T=10, cu=FAKE, table=FAKE, width=9, lens=FAKE, n=3, heads=8, max_len=100,
                           rules=None, scale=1.0, out=FAKE, lse=FAKE, ws=FAKE, bytes=need, bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw, status in SEQUENCES + [(dict(T=-1), ARG), (dict(cu=None), ARG), (dict(cu=FAKE + 2), ARG), (dict(out=None), ARG),
                                       (dict(out=FAKE + 4), ARG), (dict(ws=None), ARG), (dict(ws=FAKE + 16), ARG),
                                       (dict(bytes=need - 1), ARG), (dict(T=(1 << 30) + 1), UNSUPPORTED),
                                       (dict(T=1 << 28, max_len=1 << 29), UNSUPPORTED)]:
            assert call(**kw) == status, kw
        assert b"too many" in lib.engram_last_error()
        for r in BAD_RULES:
            assert call(rules=rules(**r)) == ARG, r
        empty = dict(q=None, out=None, cu=None, lens=None, table=None, ws=None, bytes=0, lse=None)
        assert call(T=0, **empty) == OK and call(n=0, **empty) == OK

    def test_shared_prefix_attention_rejects(self, lib):
        need = lib.engram_shared_prefix_attention_workspace_bytes(3, 2, 8, 2, 128, 500, 100)
        assert need > 0
        call = caller(lib.engram_shared_prefix_attention,
                      ("cache", "q", "cu", "ptable", "pwidth", "plens", "groups", "pmax", "table", "width", "lens", "n",
                       "heads", "max_len", "scale", "out", "lse", "ws", "bytes", "bad", "stream"),
                      dict(cache=cache(), q=FAKE, cu=FAKE, ptable=FAKE, pwidth=40, plens=FAKE, groups=2, pmax=500, table=FAKE,
                           width=9, lens=FAKE, n=3, heads=8, max_len=100, scale=1.0, out=FAKE, lse=FAKE, ws=FAKE, bytes=need,
                           bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw, status in SEQUENCES + [(dict(groups=0), ARG), (dict(groups=-1), ARG), (dict(pmax=-1), ARG), (dict(pwidth=0), ARG),
                                       (dict(pmax=(1 << 30) + 1), UNSUPPORTED), (dict(ptable=None), ARG), (dict(plens=None), ARG),
                                       (dict(ptable=FAKE + 2), ARG), (dict(plens=FAKE + 1), ARG), (dict(cu=None), ARG),
                                       (dict(out=None), ARG), (dict(ws=None), ARG), (dict(ws=FAKE + 128), ARG),
                                       (dict(bytes=need - 1), ARG), (dict(n=1 << 28, heads=8), UNSUPPORTED)]:
            assert call(**kw) == status, kw
        assert call(n=0, q=None, out=None, ws=None, bytes=0, cu=None, lens=None) == OK

    def test_cache_weights_rejects(self, lib):
        call = caller(lib.engram_cache_weights,
                      ("cache", "q", "T", "cu", "table", "width", "lens", "n", "heads", "max_len", "rules", "scale", "lse",
                       "w", "stride", "bad", "stream"),
                      dict(cache=cache(), q=FAKE, T=10, cu=FAKE, table=FAKE, width=9, lens=FAKE, n=3, heads=8, max_len=100,
                           rules=None, scale=1.0, lse=FAKE, w=FAKE, stride=100, bad=None, stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw, status in SEQUENCES + [(dict(T=-1), ARG), (dict(cu=None), ARG), (dict(lse=None), ARG), (dict(w=None), ARG),
                                       (dict(w=FAKE + 2), ARG), (dict(stride=99), ARG), (dict(stride=-1), ARG),
                                       (dict(T=1 << 29), UNSUPPORTED), (dict(n=1 << 20, max_len=1 << 20, stride=1 << 20), UNSUPPORTED)]:
            assert call(**kw) == status, kw
        for r in BAD_RULES:
            assert call(rules=rules(**r)) == ARG, r
        assert call(T=0, q=None, cu=None, lens=None, w=None) == OK and call(n=0, q=None, cu=None) == OK

    def test_cache_evict_rejects(self, lib):
        call = caller(lib.engram_cache_evict,
                      ("cache", "table", "width", "lens", "n", "max_len", "keep", "sinks", "recent", "w", "stride", "to",
                       "to_width", "new_lens", "new_w", "new_stride", "kept", "bad", "stream"),
                      dict(cache=cache(), table=FAKE, width=9, lens=FAKE, n=3, max_len=100, keep=64, sinks=4, recent=16, w=FAKE,
                           stride=100, to=FAKE, to_width=4, new_lens=FAKE, new_w=FAKE, new_stride=64, kept=FAKE, bad=None,
                           stream=None))
        for c, status in BAD_CACHES:
            assert call(cache=c) == status
        for kw in (dict(n=-1), dict(max_len=-1), dict(width=-1), dict(to_width=-1), dict(keep=-1), dict(sinks=-1),
                   dict(recent=-1), dict(sinks=60), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(to_width=3),
                   dict(stride=99), dict(new_stride=63), dict(lens=None), dict(table=None), dict(to=None), dict(w=None),
                   dict(new_lens=None), dict(new_w=None), dict(kept=None), dict(kept=FAKE + 2), dict(to=FAKE + 2),
                   dict(new_lens=FAKE + 1), dict(new_w=FAKE + 2), dict(w=FAKE + 2), dict(bad=FAKE + 1)):
            assert call(**kw) == ARG, kw
        assert call(max_len=(1 << 30) + 1, stride=1 << 31) == UNSUPPORTED
        assert call(n=1 << 26) == UNSUPPORTED
        assert call(n=0, table=None, lens=None, to=None, w=None, kept=None, new_w=None, new_lens=None) == OK

    def test_workspace_bytes(self, lib):
        chunk, shared = lib.engram_chunk_attention_workspace_bytes, lib.engram_shared_prefix_attention_workspace_bytes
        for bad in ((0, 1, 8, 2, 128, 9), (5, 0, 8, 2, 128, 9), (5, 1, 9, 2, 128, 9), (5, 1, 8, 0, 128, 9), (5, 1, 8, 2, 40, 9),
                    (5, 1, 8, 2, 128, -1), (1 << 30, 1 << 30, 8, 2, 128, 1 << 30)):
            assert chunk(*bad) == 0, bad
        assert shared(0, 1, 8, 2, 128, 9, 9) == shared(5, 0, 8, 2, 128, 9, 9) == shared(5, 1, 8, 2, 128, -1, 9) == 0
        assert chunk(1, 1, 8, 2, 128, 0) > 0
        # Short contexts are never split: no parts.
        assert chunk(64, 64, 8, 2, 128, 512) < 1 << 16 < chunk(64, 64, 8, 2, 128, 5000)


@pytest.mark.skipif(not NO_GPU, reason="the rejection cases run only without a GPU")
def test_validation_under_address_and_ub_sanitizers():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_engram_build_sanitized", os.path.join(base.ROOT, "gram_hash_memory_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    sanitized = b.build_sanitized()
    env = dict(os.environ, LD_PRELOAD=b.sanitizer_runtime(), ENGRAM_ABI_SANITIZED_LIB=sanitized,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=24")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__), "-k", "TestValidation"],
                         cwd=base.ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
