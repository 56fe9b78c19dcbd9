"""The C ABI library builds, loads and exports every entry point of
include/ksa.h; host-side validation rejects bad arguments before touching the
device.  Runs without a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared_functions():
    text = open(os.path.join(ROOT, "include", "ksa.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ksa_[a-z_0-9]+)\s*\(", text)))


@pytest.fixture(scope="module")
def ksa():
    from block_top_sparse_ksa_b200 import build
    build.build()
    import block_top_sparse_ksa_b200 as k
    return k


def test_header_declares_the_hot_path():
    names = declared_functions()
    for n in ("ksa_build_block_summaries", "ksa_select_blocks", "ksa_sparse_decode_attn",
              "ksa_unified_select"):
        assert n in names


def test_library_exports_every_declared_symbol(ksa):
    lib = ctypes.CDLL(ksa.library_path)
    missing = [n for n in declared_functions() if not hasattr(lib, n)]
    assert not missing, missing


def test_binding_wraps_every_entry_point(ksa):
    for n in declared_functions():
        assert hasattr(ksa, n), n


def test_status_strings_and_version(ksa):
    assert ksa.ksa_status_string(0) == "KSA_OK"
    assert ksa.ksa_status_string(2) == "KSA_ERR_UNSUPPORTED"
    assert ksa.ksa_version() >= 100


def _shape(ksa, B=1, Hq=4, Hkv=2, D=128, T=64, bs=16):
    return ksa.Shape(B, Hq, Hkv, D, T, bs)


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first


def test_validation_rejects_bad_shapes(ksa):
    lib = ksa.lib()
    assert lib.ksa_select_blocks(None, FAKE, FAKE, FAKE, 4, FAKE, FAKE, None, 0, None, None) == 1
    for kw, want in [(dict(D=96), 2), (dict(Hq=3, Hkv=2), 1), (dict(bs=8), 2), (dict(B=0), 1)]:
        sh = _shape(ksa, **kw)
        st = lib.ksa_select_blocks(ctypes.byref(sh), FAKE, FAKE, FAKE, 4, FAKE, FAKE, None, 0,
                                   None, None)
        assert st == want, (kw, st, ksa.ksa_last_error())
        assert ksa.ksa_last_error() != ""


def test_validation_rejects_bad_arguments(ksa):
    lib = ksa.lib()
    sh = _shape(ksa)
    # k_blocks < 1
    assert lib.ksa_select_blocks(ctypes.byref(sh), FAKE, FAKE, FAKE, 0, FAKE, FAKE, None, 0,
                                 None, None) == 1
    # NULL output
    assert lib.ksa_select_blocks(ctypes.byref(sh), FAKE, FAKE, FAKE, 4, None, FAKE, None, 0,
                                 None, None) == 1
    # summaries mode out of range
    assert lib.ksa_build_block_summaries(ctypes.byref(sh), FAKE, FAKE, 7, FAKE, None, None) == 1
    # attention: G = 16 unsupported, tokens_per_idx not a power of two, bad dtype
    sh16 = _shape(ksa, Hq=32, Hkv=2)
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh16), FAKE, FAKE, FAKE, FAKE, None, None, 0,
                                      1, 0, 0.0, 0, FAKE, None, None, 0, None, None) == 2
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 3,
                                      0, 0.0, 0, FAKE, None, None, 0, None, None) == 2
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh), FAKE, FAKE, FAKE, FAKE, None, None, 0, 1,
                                      0, 0.0, 5, FAKE, None, None, 0, None, None) == 1
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh), FAKE, FAKE, FAKE, FAKE, None, None, 0, 1,
                                      0, -1.0, 0, FAKE, None, None, 0, None, None) == 1
    # unified: recent > budget, budget > capacity, missing workspace
    assert lib.ksa_unified_select(ctypes.byref(sh), FAKE, FAKE, FAKE, 8, 16, 17, FAKE, FAKE, FAKE,
                                  1 << 20, None, None) == 1
    assert lib.ksa_unified_select(ctypes.byref(sh), FAKE, FAKE, FAKE, 8, 65, 1, FAKE, FAKE, FAKE,
                                  1 << 20, None, None) == 1
    assert lib.ksa_unified_select(ctypes.byref(sh), FAKE, FAKE, FAKE, 8, 16, 4, FAKE, FAKE, None,
                                  0, None, None) == 3


def test_workspace_sizes(ksa):
    lib = ksa.lib()
    sh = _shape(ksa, B=16, Hq=32, Hkv=8, D=128, T=20000)
    ws = lib.ksa_unified_select_workspace(ctypes.byref(sh), 4000, 4000)
    assert ws >= 16 * 32 * 20000 * 4 + 16 * 20000 * 4
    sh16 = _shape(ksa, B=32, Hq=32, Hkv=8, D=128, T=32768, bs=16)
    assert lib.ksa_select_blocks_workspace(ctypes.byref(sh16), 128) >= 32 * 8 * 2048 * 4 + 32 * 8 * 4
    assert lib.ksa_sparse_decode_attn_workspace(ctypes.byref(sh16), 128, 16) >= 32 * 8 * 4
    bad = _shape(ksa, D=96)
    assert lib.ksa_select_blocks_workspace(ctypes.byref(bad), 8) == 0


def test_missing_workspace_is_rejected(ksa):
    lib = ksa.lib()
    sh = _shape(ksa)
    assert lib.ksa_select_blocks(ctypes.byref(sh), FAKE, FAKE, FAKE, 4, FAKE, FAKE, None, 0, None,
                                 None) == 3
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh), FAKE, FAKE, FAKE, FAKE, None, None, 0, 1,
                                      0, 0.0, 0, FAKE, None, None, 0, None, None) == 3


def test_validation_of_the_newer_entry_points(ksa):
    """Storage type, window, per-head top-k, paged caches and list layouts are checked on the
    host before any device work."""
    lib = ksa.lib()
    sh = _shape(ksa)
    BIG = 1 << 30
    # summary storage type out of range
    assert lib.ksa_build_block_summaries_ex(ctypes.byref(sh), FAKE, FAKE, 0, 7, FAKE, None,
                                            None) == 1
    assert lib.ksa_select_blocks_ex(ctypes.byref(sh), FAKE, FAKE, 3, FAKE, 4, FAKE, FAKE, FAKE,
                                    BIG, None, None) == 1
    # fp8 summaries (2) need head_dim 128
    sh64 = _shape(ksa, D=64)
    assert lib.ksa_build_block_summaries_ex(ctypes.byref(sh64), FAKE, FAKE, 0, 2, FAKE, None,
                                            None) == 2
    assert lib.ksa_select_blocks_ex(ctypes.byref(sh64), FAKE, FAKE, 2, FAKE, 4, FAKE, FAKE, FAKE,
                                    BIG, None, None) == 2
    # window: k < 1, NULL output, unsupported block size
    assert lib.ksa_select_window(ctypes.byref(sh), FAKE, 0, FAKE, FAKE, None, None) == 1
    assert lib.ksa_select_window(ctypes.byref(sh), FAKE, 4, None, FAKE, None, None) == 1
    assert lib.ksa_select_window(ctypes.byref(_shape(ksa, bs=8)), FAKE, 4, FAKE, FAKE, None,
                                 None) == 2
    # per-head top-k: k < 1, G > 8, capacity above 65536
    assert lib.ksa_select_tokens_per_head(ctypes.byref(sh), FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE,
                                          BIG, None, None) == 1
    assert lib.ksa_select_tokens_per_head(ctypes.byref(_shape(ksa, Hq=32, Hkv=2)), FAKE, FAKE,
                                          FAKE, 4, FAKE, FAKE, FAKE, BIG, None, None) == 2
    assert lib.ksa_select_tokens_per_head(ctypes.byref(_shape(ksa, T=70000)), FAKE, FAKE, FAKE, 4,
                                          FAKE, FAKE, FAKE, BIG, None, None) == 2
    # paged caches: no pages, capacity != max_blocks * block_size, empty pool
    assert lib.ksa_build_block_summaries_paged(ctypes.byref(sh), FAKE, None, FAKE, 0, 0, FAKE,
                                               None, None) == 1
    bad_cap = ksa.Pages(FAKE, 3, 10)  # 3 * 16 != 64
    assert lib.ksa_build_block_summaries_paged(ctypes.byref(sh), FAKE, ctypes.byref(bad_cap),
                                               FAKE, 0, 0, FAKE, None, None) == 1
    no_pages = ksa.Pages(FAKE, 4, 0)
    assert lib.ksa_build_block_summaries_paged(ctypes.byref(sh), FAKE, ctypes.byref(no_pages),
                                               FAKE, 0, 0, FAKE, None, None) == 1
    assert lib.ksa_decode_select_blocks_paged(ctypes.byref(sh), FAKE, FAKE, ctypes.byref(bad_cap),
                                              FAKE, 0, FAKE, 4, FAKE, FAKE, FAKE, BIG, None,
                                              None) == 1
    # attention list layout out of range
    assert lib.ksa_sparse_decode_attn(ctypes.byref(sh), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 1,
                                      3, 0.0, 0, FAKE, None, None, 0, None, None) == 1


def test_sizes_past_32_bit_row_indices_are_refused(ksa):
    """K/V row coordinates are 32-bit on the device: caches of 2^31 rows or more, and page
    pools of that size, are refused on the host (KSA_ERR_UNSUPPORTED), never run."""
    lib = ksa.lib()
    big = _shape(ksa, B=1024, Hq=16, Hkv=8, T=1 << 18, bs=16)  # 1024 * 8 * 2^18 = 2^31 rows
    assert lib.ksa_select_blocks(ctypes.byref(big), FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE,
                                 1 << 30, None, None) == 2
    assert lib.ksa_sparse_decode_attn(ctypes.byref(big), FAKE, FAKE, FAKE, FAKE, None, None, 0,
                                      1, 0, 0.0, 0, FAKE, None, None, 0, None, None) == 2
    assert lib.ksa_select_blocks_workspace(ctypes.byref(big), 4) == 0
    just_under = _shape(ksa, B=1023, Hq=16, Hkv=8, T=1 << 18, bs=16)
    assert lib.ksa_select_blocks_workspace(ctypes.byref(just_under), 4) > 0
    sh = _shape(ksa, B=1, Hq=4, Hkv=2, D=128, T=64, bs=16)
    pool = ksa.Pages(FAKE, 4, 1 << 26)  # 2^26 pages * 2 kv-heads * 16 rows = 2^31
    assert lib.ksa_sparse_decode_attn_paged(ctypes.byref(sh), FAKE, FAKE, FAKE,
                                            ctypes.byref(pool), FAKE, FAKE, FAKE, 4, 16, 0, 0.0,
                                            0, FAKE, None, FAKE, 1 << 30, None, None) == 2


C_CALLER = r"""
#include <stdio.h>
#include <string.h>
#include "ksa.h"

int main(void) {
  ksa_shape sh;
  ksa_status st;
  memset(&sh, 0, sizeof sh);
  if (ksa_version() < 100) return 1;
  if (strcmp(ksa_status_string(KSA_ERR_UNSUPPORTED), "KSA_ERR_UNSUPPORTED") != 0) return 2;
  /* a NULL shape and an empty batch are refused on the host, with a message */
  st = ksa_select_blocks(NULL, NULL, NULL, NULL, 4, NULL, NULL, NULL, 0, NULL, NULL);
  if (st != KSA_ERR_INVALID_ARG || ksa_last_error()[0] == '\0') return 3;
  sh.batch = 0; sh.num_q_heads = 4; sh.num_kv_heads = 2; sh.head_dim = 128;
  sh.capacity = 64; sh.block_size = 16;
  st = ksa_sparse_decode_attn(&sh, NULL, NULL, NULL, NULL, NULL, NULL, 0, 1, KSA_IDX_PER_KV_HEAD,
                              0.0f, KSA_OUT_F32, NULL, NULL, NULL, 0, NULL, NULL);
  if (st != KSA_ERR_INVALID_ARG) return 4;
  sh.batch = 2;
  if (ksa_select_blocks_workspace(&sh, 4) == 0) return 5;
  printf("ok %d\n", (int)ksa_version());
  return 0;
}
"""


@pytest.mark.parametrize("lang", ["c99", "c++11"])
def test_c_caller_builds_links_and_runs(ksa, tmp_path, lang):
    """A plain C (and C++) program includes include/ksa.h, links libksa.so and makes the
    host-only calls: version, status strings, validation errors, workspace sizes."""
    import shutil
    import subprocess
    src = tmp_path / ("caller.c" if lang == "c99" else "caller.cpp")
    src.write_text(C_CALLER)
    exe = tmp_path / "caller"
    libdir = os.path.dirname(ksa.library_path)
    cc = "gcc" if lang == "c99" else "g++"
    if shutil.which(cc) is None:
        pytest.skip(f"{cc} not found")
    cmd = [cc, f"-std={lang}", "-Wall", "-Wextra", "-Werror", "-pedantic",
           "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
           "-L", libdir, "-l:" + os.path.basename(ksa.library_path), "-Wl,-rpath," + libdir]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, (out.returncode, out.stderr)
    assert out.stdout.startswith("ok ")


def test_no_fallback_without_the_library_or_a_gpu(tmp_path):
    """The product path has no CPU fallback: CPU tensors are refused before any call, and a
    missing library is an error naming the build step (checked in a fresh interpreter)."""
    import subprocess
    import sys
    code = (
        "import sys, torch\n"
        f"sys.path.insert(0, {ROOT!r})\n"
        "import block_top_sparse_ksa_b200 as k\n"
        "q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)\n"
        "K = torch.zeros((1, 2, 64, 128), dtype=torch.bfloat16)\n"
        "L = torch.full((1,), 64, dtype=torch.int32)\n"
        "try:\n"
        "    k.ksa_sparse_decode_attn(q, K, K, L)\n"
        "    sys.exit('CPU tensors were accepted')\n"
        "except TypeError as e:\n"
        "    assert 'CUDA tensor' in str(e), e\n"
        f"k.library_path = {str(tmp_path / 'libksa_absent.so')!r}\n"
        "k._LIB = None\n"
        "try:\n"
        "    k.lib()\n"
        "    sys.exit('a missing library loaded')\n"
        "except RuntimeError as e:\n"
        "    assert 'missing' in str(e) and 'build' in str(e), e\n"
        "print('ok')\n")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.strip().endswith("ok")


def test_validation_of_random_head_selection(ksa):
    """The host array of heads is checked row by row before any launch."""
    lib = ksa.lib()
    sh = _shape(ksa, B=3, Hq=8, Hkv=2)
    good = (ctypes.c_int32 * 3)(0, 7, 3)
    bad = (ctypes.c_int32 * 3)(0, 8, 3)  # head 8 of 8
    neg = (ctypes.c_int32 * 3)(-1, 0, 0)
    BIG = 1 << 30
    call = lambda heads, k, ws, n: lib.ksa_select_tokens_one_head(
        ctypes.byref(sh), FAKE, FAKE, FAKE, heads, k, FAKE, FAKE, ws, n, None, None)
    assert call(None, 4, FAKE, BIG) == 1
    assert call(bad, 4, FAKE, BIG) == 1 and "head_of_row[1]" in ksa.ksa_last_error()
    assert call(neg, 4, FAKE, BIG) == 1
    assert call(good, 0, FAKE, BIG) == 1
    assert call(good, 4, None, 0) == 3
    per_head = lib.ksa_select_tokens_per_head_workspace(ctypes.byref(sh), 4)
    one_head = lib.ksa_select_tokens_one_head_workspace(ctypes.byref(sh), 4)
    assert one_head >= per_head + 3 * 8 * 4 * 4 + 3 * 8 * 4 + 3 * 4  # lists, counts, heads
    assert call(good, 4, FAKE, one_head - 1) == 3


def test_every_entry_point_refuses_a_null_shape(ksa):
    """Driven by the binding's signature table: each call that takes a shape first returns
    KSA_ERR_INVALID_ARG (status calls) or 0 bytes (workspace queries) for a NULL shape, with
    every other pointer NULL and every number 0 -- validation first, nothing dereferenced."""
    lib = ksa.lib()
    checked = 0
    for name, (res, args) in ksa._SIGS.items():
        if not args or args[0] is not ctypes.POINTER(ksa.Shape):
            continue
        rest = []
        for t in args[1:]:
            if t in (ctypes.c_float, ctypes.c_double):
                rest.append(0.0)
            elif t in (ctypes.c_int32, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint32):
                rest.append(0)
            else:
                rest.append(None)
        got = getattr(lib, name)(None, *rest)
        want = 0 if res is ctypes.c_size_t else 1
        assert got == want, (name, got)
        checked += 1
    assert checked >= 20


def test_device_status_read_back_validation(ksa):
    lib = ksa.lib()
    flags = ctypes.c_uint32(7)
    assert lib.ksa_get_device_status(None, None, 0, ctypes.byref(flags)) == 1
    assert lib.ksa_get_device_status(FAKE, None, 0, None) == 1
    assert flags.value == 7  # untouched on a refused call


# The one kernel allowed a spill: the token-list attention at head_dim 128 runs two producer
# warps, so three CTAs of six warps hold at most 96 registers a thread (five warps of one
# sub-partition share its 16K registers), and it spills a few words; measured against the
# one-producer form without spills it is faster (65.5 -> 59.9 us per LessIsMore layer).
SPILL_ALLOWED = {"sparse_decode_attn_kernelILi128ELi2E": 64}  # kernel -> max bytes


def test_no_kernel_spills_registers(ksa):
    """The last build's ptxas report: every kernel fits its registers (the selection and pick
    kernels keep whole rows of keys in registers; a spill would send them to local memory),
    but for the listed one, within its bound."""
    from block_top_sparse_ksa_b200 import build
    if not os.path.exists(build.REPORT):
        build.build(force=True)
    text = open(build.REPORT).read()
    blocks = re.split(r"Compiling entry function '", text)[1:]
    assert len(blocks) >= 30
    for blk in blocks:
        name = blk.split("'", 1)[0]
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", blk)
        assert m, name
        allowed = max([v for k, v in SPILL_ALLOWED.items() if k in name], default=0)
        assert int(m.group(1)) <= allowed and int(m.group(2)) <= allowed, (name, m.groups())


def test_validation_of_the_decode_step_and_append(ksa):
    """ksa_decode_step checks the arguments of both calls it stands for, then its own
    workspace; ksa_append_kv checks pointers and alignment.  Nothing reaches the device."""
    lib = ksa.lib()
    sh = _shape(ksa, B=2, Hq=8, Hkv=2, D=128, T=256, bs=16)
    args = lambda **kw: [kw.get("q", FAKE), kw.get("K", FAKE), FAKE, FAKE, 0, FAKE,
                         kw.get("k", 8), FAKE, FAKE, kw.get("scale", 0.0), 0, FAKE, None,
                         kw.get("ws", None), kw.get("ws_bytes", 0), None, None]
    assert lib.ksa_decode_step(None, *args()) == 1
    assert lib.ksa_decode_step(ctypes.byref(sh), *args(K=None)) == 1
    assert lib.ksa_decode_step(ctypes.byref(sh), *args(k=0)) == 1
    assert lib.ksa_decode_step(ctypes.byref(sh), *args(scale=-1.0)) == 1
    assert lib.ksa_decode_step(ctypes.byref(sh), *args()) == 3  # no workspace
    need = lib.ksa_decode_step_workspace(ctypes.byref(sh), 8)
    assert need >= (lib.ksa_select_blocks_workspace(ctypes.byref(sh), 8) +
                    lib.ksa_sparse_decode_attn_workspace(ctypes.byref(sh), 8, 16))
    assert lib.ksa_decode_step(ctypes.byref(sh), *args(ws=FAKE, ws_bytes=need - 1)) == 3
    bad = _shape(ksa, B=2, Hq=8, Hkv=2, D=128, T=256, bs=8)
    assert lib.ksa_decode_step(ctypes.byref(bad), *args()) == 2
    assert lib.ksa_append_kv(ctypes.byref(sh), FAKE, None, FAKE, FAKE, FAKE, None, None) == 1
    odd = ctypes.c_void_p(0x1008)  # 8-byte aligned only
    assert lib.ksa_append_kv(ctypes.byref(sh), odd, FAKE, FAKE, FAKE, FAKE, None, None) == 1
    assert "aligned" in ksa.ksa_last_error()


def test_validation_of_page_assignment_and_release(ksa):
    lib = ksa.lib()
    sh = _shape(ksa, B=2, T=64, bs=16)
    BIG = 1 << 20

    def assign(**kw):
        a = dict(sh=sh, ctx=FAKE, new=FAKE, table=FAKE, mb=4, pages=9, free=FAKE, nf=FAKE,
                 nfo=FAKE, n=5, seq=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, ws=FAKE, wsb=BIG)
        a.update(kw)
        return lib.ksa_assign_pages(ctypes.byref(a["sh"]), a["ctx"], a["new"], a["table"],
                                    a["mb"], a["pages"], a["free"], a["nf"], a["nfo"], a["n"],
                                    a["seq"], a["cu"], a["slots"], a["pos"], a["ws"], a["wsb"],
                                    None, None)

    for kw in (dict(ctx=None), dict(new=None), dict(table=None), dict(free=None), dict(nf=None),
               dict(nfo=None), dict(seq=None), dict(cu=None), dict(slots=None), dict(pos=None),
               dict(mb=0), dict(mb=3), dict(pages=0), dict(n=-1), dict(n=1 << 30),
               dict(slots=ctypes.c_void_p(0x1004)), dict(ctx=ctypes.c_void_p(0x1002))):
        assert assign(**kw) == 1, kw
        assert ksa.ksa_last_error() != ""
    assert assign(sh=_shape(ksa, bs=8)) == 2
    far = (1 << 26) + 1  # blocks of 16: 2^30 + 16 tokens
    assert assign(sh=_shape(ksa, B=1, Hq=1, Hkv=1, T=far * 16), mb=far) == 2
    for kw in (dict(ws=None), dict(wsb=255), dict(ws=ctypes.c_void_p(0x1010))):
        assert assign(**kw) == 3, kw

    def release(**kw):
        a = dict(done=FAKE, seq=FAKE, table=FAKE, mb=4, pages=9, free=FAKE, nf=FAKE, ws=FAKE)
        a.update(kw)
        return lib.ksa_release_pages(ctypes.byref(sh), a["done"], a["seq"], a["table"], a["mb"],
                                     a["pages"], a["free"], a["nf"], a["ws"], BIG, None, None)

    for kw in (dict(done=None), dict(seq=None), dict(table=None), dict(mb=5), dict(pages=0),
               dict(free=None), dict(nf=None)):
        assert release(**kw) == 1, kw
    assert release(ws=None) == 3


def test_validation_of_rotary_appends(ksa):
    """The rotation's tables are checked entry by entry on the host; pointers come in groups;
    strides hold the heads and keep 16-byte chunks."""
    lib = ksa.lib()
    sh = _shape(ksa, B=1, Hq=4, Hkv=2, D=128, T=64, bs=16)
    good = ksa.Rotary([0.5] * 64)

    def call(rot=good, paged=False, **kw):
        a = dict(sh=sh, n=3, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, slots=FAKE,
                 qo=FAKE, qos=512, K=FAKE, V=FAKE, pages=4)
        a.update(kw)
        args = [ctypes.byref(a["sh"]), a["n"], rot._ref if rot is not None else None, a["q"],
                a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["slots"], a["qo"],
                a["qos"], a["K"], a["V"]]
        if paged:
            return lib.ksa_rotary_append_kv_paged(*args, a["pages"], None, None)
        return lib.ksa_rotary_append_kv(*args, None, None)

    odd = ctypes.c_void_p(0x1008)
    for kw in (dict(n=-1), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(K=None),
               dict(V=None), dict(slots=None), dict(pos=None), dict(q=odd), dict(K=odd),
               dict(qs=511), dict(qs=516), dict(qs=504), dict(ks=248), dict(vs=250), dict(qos=8),
               dict(rot=None), dict(qos=520),
               dict(q=None, qo=None, k=None, v=None, K=None, V=None),
               dict(rot=ksa.Rotary([0.5] * 4)), dict(rot=ksa.Rotary([0.5] * 9)),
               dict(rot=ksa.Rotary([0.5] * 72)), dict(rot=ksa.Rotary([])),
               dict(rot=ksa.Rotary([0.5] * 63 + [float("inf")])),
               dict(rot=ksa.Rotary([float("nan")] * 64)),
               dict(rot=ksa.Rotary([0.5] * 64, [0] * 63 + [2], num_axes=2)),
               dict(rot=ksa.Rotary([0.5] * 64, [-1] + [0] * 63, num_axes=2)),
               dict(rot=ksa.Rotary([0.5] * 64, num_axes=9)),
               dict(paged=True, pages=0)):
        assert call(**kw) == 1, kw
        assert ksa.ksa_last_error() != ""
    assert call(paged=True, pages=1 << 27) == 2
    assert call(paged=True, sh=_shape(ksa, bs=8)) == 2
    assert call(sh=_shape(ksa, D=96)) == 2
    assert call(n=0, q=None) == 0  # nothing to do
    with pytest.raises(ValueError):
        ksa.Rotary([0.5] * 64, [0] * 3)


def test_validation_of_chunk_attention(ksa):
    lib = ksa.lib()
    sh = _shape(ksa, B=2, Hq=4, Hkv=2, D=128, T=64, bs=16)
    need = lib.ksa_chunk_attn_workspace(ctypes.byref(sh), 7)
    assert need >= 256 and need % 256 == 0
    pages = ksa.Pages(FAKE, 4, 10)

    def call(paged=False, **kw):
        a = dict(sh=sh, n=7, q=FAKE, qs=512, K=FAKE, V=FAKE, cu=FAKE, seq=FAKE, mask=1, scale=0.0,
                 out=FAKE, lse=None, ws=FAKE, wsb=need, pages=ctypes.byref(pages))
        a.update(kw)
        rest = [a["cu"], a["seq"], a["mask"], a["scale"], a["out"], a["lse"], a["ws"], a["wsb"],
                None, None]
        args = [ctypes.byref(a["sh"]), a["n"], a["q"], a["qs"], a["K"], a["V"]]
        if paged:
            return lib.ksa_chunk_attn_paged(*args, a["pages"], *rest)
        return lib.ksa_chunk_attn(*args, *rest)

    odd = ctypes.c_void_p(0x1008)
    for kw in (dict(n=-1), dict(q=None), dict(K=None), dict(V=None), dict(cu=None), dict(seq=None),
               dict(out=None), dict(q=odd), dict(V=odd), dict(out=odd), dict(mask=2),
               dict(mask=-1), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(qs=504), dict(qs=516),
               dict(lse=ctypes.c_void_p(0x1002)), dict(paged=True, pages=None),
               dict(paged=True, pages=ctypes.byref(ksa.Pages(FAKE, 3, 10))),
               dict(paged=True, pages=ctypes.byref(ksa.Pages(FAKE, 4, 0)))):
        assert call(**kw) == 1, kw
        assert ksa.ksa_last_error() != ""
    for kw in (dict(ws=None), dict(wsb=need - 1), dict(ws=ctypes.c_void_p(0x1010))):
        assert call(**kw) == 3, kw
    assert call(sh=_shape(ksa, Hq=258, Hkv=2)) == 2
    assert call(sh=_shape(ksa, D=96)) == 2
    assert call(paged=True, sh=_shape(ksa, bs=8)) == 2
    assert call(n=1 << 30) == 2
    assert call(sh=_shape(ksa, B=1, Hq=1, Hkv=1, T=(1 << 30) + 1), qs=128) == 2
    assert call(n=0, q=None) == 0
    bad = _shape(ksa, D=96)
    assert lib.ksa_chunk_attn_workspace(ctypes.byref(bad), 7) == 0


def test_serving_calls_refuse_cpu_tensors(ksa):
    """The tensors' type, shape and device are checked before the library is called; CPU tensors
    are refused by name."""
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="block_table must be a CUDA tensor"):
        ksa.ksa_assign_pages(i32(2), i32(2), i32(2, 4), i32(9), i32(1), 16, 3)
    with pytest.raises(TypeError, match="block_table must be a CUDA tensor"):
        ksa.ksa_release_pages(i32(2), i32(2), i32(2, 4), i32(9), i32(1), 16)
    rot = ksa.Rotary([0.5] * 64)
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        ksa.ksa_rotary_append_kv(bf(3, 4, 128), bf(3, 2, 128), bf(3, 2, 128), i32(3),
                                 torch.zeros(3, dtype=torch.int64), bf(1, 2, 8, 128),
                                 bf(1, 2, 8, 128), rot)
    with pytest.raises(ValueError, match="together"):
        ksa.ksa_rotary_append_kv(bf(3, 4, 128), bf(3, 2, 128), None, i32(3), None, None, None, rot)
    with pytest.raises(ValueError, match="Rotary"):
        ksa.ksa_rotary_append_kv(bf(3, 4, 128), None, None, i32(3), None, None, None, None)
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        ksa.ksa_chunk_attn(bf(3, 4, 128), bf(1, 2, 8, 128), bf(1, 2, 8, 128), i32(2), i32(1))
    with pytest.raises(TypeError, match="block_table must be a CUDA tensor"):
        ksa.ksa_chunk_attn_paged(bf(3, 4, 128), bf(1, 2, 16, 128), bf(1, 2, 16, 128), None,
                                 i32(2), i32(1))


def test_serving_calls_refuse_an_unaligned_status_word(ksa):
    """An atomic on a word that is not 4-byte aligned would fault: refused by every serving
    call."""
    lib = ksa.lib()
    odd = ctypes.c_void_p(0x1002)
    sh = _shape(ksa, B=2, Hq=4, Hkv=2, D=128, T=64, bs=16)
    ref, big = ctypes.byref(sh), 1 << 30
    pages = ksa.Pages(FAKE, 4, 10)
    rot = ksa.Rotary([1.0] * 64)._ref
    calls = [
        lambda s: lib.ksa_assign_pages(ref, FAKE, FAKE, FAKE, 4, 9, FAKE, FAKE, FAKE, 5, FAKE,
                                       FAKE, FAKE, FAKE, FAKE, big, s, None),
        lambda s: lib.ksa_release_pages(ref, FAKE, FAKE, FAKE, 4, 9, FAKE, FAKE, FAKE, big, s,
                                        None),
        lambda s: lib.ksa_rotary_append_kv(ref, 3, rot, FAKE, 512, FAKE, 256, FAKE, 256, FAKE,
                                           FAKE, FAKE, 512, FAKE, FAKE, s, None),
        lambda s: lib.ksa_rotary_append_kv_paged(ref, 3, rot, FAKE, 512, FAKE, 256, FAKE, 256,
                                                 FAKE, FAKE, FAKE, 512, FAKE, FAKE, 10, s, None),
        lambda s: lib.ksa_chunk_attn(ref, 7, FAKE, 512, FAKE, FAKE, FAKE, FAKE, 1, 0.0, FAKE,
                                     None, FAKE, big, s, None),
        lambda s: lib.ksa_chunk_attn_paged(ref, 7, FAKE, 512, FAKE, FAKE, ctypes.byref(pages),
                                           FAKE, FAKE, 1, 0.0, FAKE, None, FAKE, big, s, None),
    ]
    for call in calls:
        assert call(odd) == 1
        assert "dev_status" in ksa.ksa_last_error()


def test_short_way_of_the_serving_calls(ksa):
    """The binding's compiled argument checks are built with the library; what does not match
    (CPU tensors, missing outputs, wrong types and numbers) is left to the Python checks."""
    import torch
    ksa.lib()
    m = ksa._marshal
    assert m is not None and set(ksa._ENTRIES) == set(ksa._SHORT) and all(ksa._ENTRIES.values())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ws, slots = torch.zeros(256, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    e = ksa._ENTRIES["ksa_assign_pages"]
    assign = [e, i32(2), i32(2), i32(2, 4), i32(9), i32(1), 16, 3, None, i32(2), i32(3), slots,
              i32(3), ws, None]
    assert m.assign_pages(*assign) is None  # not on a GPU
    for i in range(len(assign)):
        for bad in (None, "x", 1 << 40, -1, 0, 2.5, torch.zeros(0)):
            assert m.assign_pages(*assign[:i], bad, *assign[i + 1:]) is None
    rot = ksa.Rotary([1.0] * 64)
    args = [ksa._ENTRIES["ksa_rotary_append_kv"], False, bf(3, 4, 128), bf(3, 2, 128),
            bf(3, 2, 128), i32(3), slots, bf(1, 2, 8, 128), bf(1, 2, 8, 128), rot._address,
            bf(3, 4, 128), None]
    assert m.rotary_append(*args) is None
    attn = [ksa._ENTRIES["ksa_chunk_attn"], bf(3, 4, 128), bf(1, 2, 8, 128), bf(1, 2, 8, 128),
            None, i32(2), i32(1), 1, 0.0, bf(3, 4, 128), None, ws, None]
    assert m.chunk_attn(*attn) is None
    for f, a in ((m.assign_pages, assign), (m.rotary_append, args), (m.chunk_attn, attn),
                 (m.release_pages, [None] * 9)):
        with pytest.raises(TypeError, match="number of arguments"):
            f(*a[:-1])
    assert m.release_pages(*[None] * 9) is None


def test_chunk_attention_waits_end_for_whole_warps():
    """A wait that gives up must end for all lanes of its warp alike: the others would wait for
    ever at the next vote.  So every wait is voted on, except the products warp's, whose lanes stay
    in step to the item's end (no lane leaves between a wait and the vote there)."""
    here = os.path.join(ROOT, "block_top_sparse_ksa_b200", "csrc", "chunk_attn.cu")
    with open(here) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.rindex("} else if (warp == kMmaWarp) {")
    products = text[at:text.index("} else if (warp < kSoftWarps) {")]
    others = text.replace(products, "")
    # the definition, and warp_wait's call under its vote
    assert len(re.findall(r"\bwait_bar\(", others)) == 2
    assert re.search(r"return __all_sync\(0xffffffffu, wait_bar\(bar, parity, abort\)\);", others)
    assert len(re.findall(r"\bwait_bar\(", products)) == 5
    assert len(re.findall(r"ok = ok && wait_bar\(", products)) == 5
    assert "break" not in products and "return false" not in products
    loops = re.findall(r"(?:for|while) \([^\n]*\bok\b[^\n]*", products)
    assert loops == ["while (ok && take.get(ctl, w) && w.token >= 0) {"]
    assert re.search(r"ok = __all_sync\(0xffffffffu, ok\);\s*}\s*mma_commit", products)


def test_library_is_built_where_the_short_way_cannot_be(ksa, tmp_path, monkeypatch, capsys):
    """A compiler that is missing or fails leaves libksa.so built and no stale _marshal.so."""
    import shutil
    from block_top_sparse_ksa_b200 import build
    real = build.LIB
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libksa.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "REPORT", str(tmp_path / "_build" / "ptxas.txt"))
    monkeypatch.setattr(build, "_lib_command", lambda: ["cp", real, build.LIB + ".tmp"])
    for command in (["false"], [str(tmp_path / "no_such_compiler")]):
        monkeypatch.setattr(build, "_marshal_command", lambda: command)
        (tmp_path / "_marshal.so").write_bytes(b"of other sources")
        assert build.build(force=True) == build.LIB
        assert os.path.exists(build.LIB) and os.path.exists(build.REPORT)
        assert not os.path.exists(build.MARSHAL) and not build.up_to_date()
        assert "_marshal.so could not be built" in capsys.readouterr().err
        os.remove(build.LIB)
    # and a library that fails to build is still an error, the marshal built or not
    monkeypatch.setattr(build, "_lib_command", lambda: ["false"])
    with pytest.raises(Exception, match="false"):
        build.build(force=True)


def test_short_way_of_another_torch_is_not_used(ksa, monkeypatch):
    """_marshal.so reads tensors by the layout of the torch it was compiled against: after torch is
    exchanged it counts as out of date, and is not used until it is built again."""
    from block_top_sparse_ksa_b200 import build
    ksa.lib()
    assert build.up_to_date() and ksa._load_marshal() is ksa._marshal
    other = lambda: "torch 9.9.9 python 3.12"
    monkeypatch.setattr(build, "built_for", other)
    assert not build.up_to_date()
    monkeypatch.setattr(ksa, "_built_for", other)
    with pytest.warns(UserWarning, match="built for torch"):
        assert ksa._load_marshal() is None


def test_serving_entries_keep_exceptions_inside():
    """No exception (out of host memory, for a message) leaves a serving call's C entry: each one's
    body runs guarded."""
    path = os.path.join(ROOT, "block_top_sparse_ksa_b200", "csrc", "ksa_api.cu")
    with open(path) as f:
        text = f.read()
    for name in ("ksa_assign_pages", "ksa_release_pages", "ksa_rotary_append_kv",
                 "ksa_rotary_append_kv_paged", "ksa_chunk_attn_workspace", "ksa_chunk_attn",
                 "ksa_chunk_attn_paged"):
        body = re.search(r"^(?:ksa_status|size_t) " + name + r"\([^{]*\{\n(.*?)^}", text,
                         re.S | re.M).group(1)
        lines = [x.strip() for x in body.splitlines() if x.strip()]
        start = next(i for i, x in enumerate(lines) if "guarded([&]() -> ksa_status {" in x)
        assert all(re.fullmatch(r"size_t \w+ = 0;", x) for x in lines[:start]), name
        end = lines.index("});")
        assert lines[end + 1:] in ([], ["return bytes;"]), name


def test_rotary_refuses_numbers_past_32_bits(ksa):
    """An axis or a number of axes past 32 bits is not cut off."""
    for kw in (dict(num_axes=(1 << 32) + 1), dict(axis_of_pair=[0] * 31 + [1 << 32])):
        with pytest.raises(ValueError, match="32 bits"):
            ksa.Rotary([0.5] * 32, **kw)
