"""Host-side checks of libvfa (no GPU): it builds, loads, exports every symbol
that include/vfa.h declares, and rejects bad arguments before touching a
device.  No call here launches a kernel."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def vfa():
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    binding.lib()
    return binding


def _declared_symbols():
    with open(os.path.join(ROOT, "include", "vfa.h")) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(vfa_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def test_exports_every_declared_symbol(vfa):
    declared = _declared_symbols()
    assert len(declared) >= 10
    L = vfa.lib()
    for name in declared:
        assert hasattr(L, name), f"{name} declared in vfa.h but not exported"
    bound = {n for n, _, _ in vfa.SIGNATURES}
    assert bound == set(declared), "binding and header disagree"


def test_version_and_tile_shape(vfa):
    assert "sm_103a" in vfa.version()
    assert vfa.tile_shape(64) == (128, 128, True)
    assert vfa.tile_shape(128) == (128, 128, True)
    assert vfa.tile_shape(256) == (128, 64, False)
    with pytest.raises(vfa.VfaError) as e:
        vfa.tile_shape(96)
    assert e.value.status == vfa.VFA_ERR_UNSUPPORTED


def test_workspace_bound_covers_worst_case(vfa):
    # one item per (q tile, head); the bound must hold for any split of total_q
    import oracle
    from variable_length_flashattention_gb300 import workloads as W
    for lengths in ([1] * 50, [129] * 7, [128, 1, 0, 255, 3], [5000]):
        cu = W.cu_seqlens(lengths)
        n_items = len(oracle.schedule(cu, cu, 3, 128, 128, True))
        total = int(cu[-1])
        ws = vfa.workspace_bytes(len(lengths), total, total, 3, 128)
        assert ws >= 256 + 32 * n_items
    assert vfa.lib().vfa_varlen_fwd_workspace_bytes(0, 10, 10, 1, 128) == 0
    assert vfa.lib().vfa_varlen_fwd_workspace_bytes(1, 10, 10, 1, 80) == 0


def test_host_rejects_null_and_unsupported(vfa):
    L = vfa.lib()
    nul = None
    st = L.vfa_varlen_fwd(nul, nul, nul, nul, nul, 1, 1, 1, 1, 1, 1, 128, 1.0, 0, -1, nul, nul, nul, 0,
                          nul)
    assert st == vfa.VFA_ERR_INVALID_ARG
    assert b"null" in L.vfa_last_error()
    fake = ctypes.c_void_p(0x100000)   # never dereferenced: rejected before any device work
    st = L.vfa_varlen_fwd(fake, fake, fake, fake, fake, 1, 1, 1, 1, 1, 1, 96, 1.0, 0, -1, fake, fake,
                          fake, 1 << 20, nul)
    assert st == vfa.VFA_ERR_UNSUPPORTED
    st = L.vfa_varlen_fwd(fake, fake, fake, fake, fake, 1, 1, 1, 1, 1, 1, 128, 1.0, 0, -1, fake, fake,
                          fake, 16, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG and b"workspace too small" in L.vfa_last_error()
    st = L.vfa_varlen_fwd(fake, fake, fake, fake, fake, 1, 1, 1, 1, 6, 4, 128, 1.0, 0, -1, fake, fake,
                          fake, 1 << 20, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG and b"num_kv_heads" in L.vfa_last_error()
    odd = ctypes.c_void_p(0x100002)
    st = L.vfa_varlen_fwd(odd, fake, fake, fake, fake, 1, 1, 1, 1, 1, 1, 128, 1.0, 0, -1, fake, fake,
                          fake, 1 << 20, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG and b"aligned" in L.vfa_last_error()
    # a sliding window without a causal mode
    st = L.vfa_varlen_fwd(fake, fake, fake, fake, fake, 1, 1, 1, 1, 1, 1, 128, 1.0, 0, 16, fake, fake,
                          fake, 1 << 20, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG and b"window" in L.vfa_last_error()
    # decode: unsupported group size / block size / head_dim
    st = L.vfa_paged_decode_step(fake, fake, fake, 4, fake, fake, nul, 2, 1, 12, 4, 128, 16, 0.0,
                                 fake, fake, fake, nul, nul)
    assert st == vfa.VFA_ERR_UNSUPPORTED
    st = L.vfa_paged_decode_step(fake, fake, fake, 4, fake, fake, nul, 2, 1, 8, 2, 128, 32, 0.0,
                                 fake, fake, fake, nul, nul)
    assert st == vfa.VFA_ERR_UNSUPPORTED
    st = L.vfa_paged_decode_step(fake, fake, fake, 4, fake, fake, nul, 2, 1, 9, 2, 128, 16, 0.0,
                                 fake, fake, fake, nul, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG
    st = L.vfa_paged_decode_step(fake, fake, fake, 4, fake, fake, nul, 2, 1, 8, 2, 128, 16,
                                 float("nan"), fake, fake, fake, nul, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG and b"softmax_scale" in L.vfa_last_error()
    st = L.vfa_paged_decode_finalize(fake, fake, 1, 1, 12, fake, nul)
    assert st == vfa.VFA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors(vfa):
    import torch
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        vfa.varlen_fwd(x, x, x, cu, cu, 4, 0.125, False)


def test_product_path_does_not_import_the_oracle():
    pkg = os.path.join(ROOT, "variable_length_flashattention_gb300")
    for dirpath, _, files in os.walk(pkg):
        for fn in files:
            if fn.endswith((".py", ".cu", ".cuh", ".h")):
                with open(os.path.join(dirpath, fn)) as f:
                    src = f.read()
                assert not re.search(r"^\s*(import|from)\s+oracle\b", src, re.M), fn
                assert "vfa_oracle" not in src, fn


def test_backward_and_fp8_host_checks(vfa):
    # rejected on the host before any device work (no GPU needed)
    L = vfa.lib()
    fake = ctypes.c_void_p(0x100000)
    nul = None
    args = lambda D, scale, causal, wl, q=fake: (q, fake, fake, fake, fake, fake, fake, fake,
                                                 4, 4, 1, 2, 2, D, scale, causal, wl, fake, fake,
                                                 fake, fake, 1 << 30, nul)
    assert L.vfa_varlen_bwd(*args(128, 0.1, 1, -1, q=nul)) == vfa.VFA_ERR_INVALID_ARG
    assert b"null" in L.vfa_last_error()
    assert L.vfa_varlen_bwd(*args(96, 0.1, 1, -1)) == vfa.VFA_ERR_UNSUPPORTED
    assert L.vfa_varlen_bwd(*args(128, 0.0, 1, -1)) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_varlen_bwd(*args(128, 0.1, 0, 8)) == vfa.VFA_ERR_INVALID_ARG
    assert b"window" in L.vfa_last_error()
    assert L.vfa_varlen_bwd(*args(128, 0.1, 3, -1)) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_varlen_bwd_workspace_bytes(1, 10, 2, 96) == 0
    assert L.vfa_varlen_bwd_workspace_bytes(1, 10, 2, 256) > 0
    # status word, key-tile and q-tile starts, Delta; no fp32 dq sum (dq is
    # accumulated in TMEM per query tile)
    assert L.vfa_varlen_bwd_workspace_bytes(2, 10, 2, 128) >= 256 + 2 * 3 * 4 + 10 * 2 * 4
    assert L.vfa_varlen_bwd_workspace_bytes(2, 10, 2, 128) < 10 * 2 * 128 * 4
    # FP8 forward: head_dim 64, 128 or 256, descales finite and positive
    f8 = lambda D, dq, dk: (fake, fake, fake, fake, fake, 4, 4, 4, 1, 2, 2, D, 0.1, dq, dk, 1, -1,
                            fake, fake, fake, 1 << 30, nul)
    assert L.vfa_varlen_fwd_fp8(*f8(96, 1.0, 1.0)) == vfa.VFA_ERR_UNSUPPORTED
    assert L.vfa_varlen_fwd_fp8(*f8(128, 0.0, 1.0)) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_varlen_fwd_fp8(*f8(128, 1.0, float("inf"))) == vfa.VFA_ERR_INVALID_ARG


def test_noalloc_rejects_problems_beyond_the_static_scratch(vfa):
    # The static scratch of vfa_varlen_fwd_noalloc holds 1 MiB; a problem whose
    # workspace is larger is refused on the host, before any device work.
    L = vfa.lib()
    nul = None
    # 100k one-token sequences x 8 heads need far more than 1 MiB of work list
    assert L.vfa_varlen_fwd_workspace_bytes(100000, 100000, 100000, 8, 128) > (1 << 20)
    st = L.vfa_varlen_fwd_noalloc(nul, nul, nul, nul, nul, 100000, 100000, 1, 100000, 8, 8, 128,
                                  0.1, 0, -1, nul, nul, nul, nul)
    assert st == vfa.VFA_ERR_UNSUPPORTED
    assert b"static scratch" in L.vfa_last_error()
    # the limit is the exact size: one work item (32 bytes) past it is refused
    r = lambda x: (x + 255) // 256 * 256
    size = lambda B, tq, H: r(r(256 + 32 * H * (tq // 128 + B)) + 56 * (B + 1))
    B, H = 1, 1
    tq = 128 * ((1 << 20) - 1024) // 32         # just inside
    while size(B, tq + 128, H) <= (1 << 20):
        tq += 128
    assert size(B, tq, H) <= (1 << 20) < size(B, tq + 128, H)
    assert L.vfa_varlen_fwd_workspace_bytes(B, tq, tq, H, 128) == size(B, tq, H)
    st = L.vfa_varlen_fwd_noalloc(nul, nul, nul, nul, nul, tq + 128, tq + 128, 1, B, H, H, 128,
                                  0.1, 0, -1, nul, nul, nul, nul)
    assert st == vfa.VFA_ERR_UNSUPPORTED
    # within the limit the call gets past the size check (and then stops at the
    # missing device or the null pointers)
    st = L.vfa_varlen_fwd_noalloc(nul, nul, nul, nul, nul, tq, tq, 1, B, H, H, 128, 0.1, 0, -1,
                                  nul, nul, nul, nul)
    assert st in (vfa.VFA_ERR_INVALID_ARG, vfa.VFA_ERR_CUDA)
    assert b"static scratch" not in L.vfa_last_error()


def test_split_decode_host_checks(vfa):
    # the split step's workspace size is exact and its arguments are checked
    # on the host before any device work (no GPU needed)
    L = vfa.lib()
    r = lambda x: (x + 255) // 256 * 256
    for S, Hq, Hkv, D, n in ((4, 32, 8, 128, 19), (1, 8, 8, 64, 1), (64, 32, 8, 256, 1024)):
        want = r(r(S * Hkv * 4) + S * Hq * n * (D + 2) * 4)
        assert L.vfa_paged_decode_split_workspace_bytes(S, Hq, Hkv, D, n) == want
    # unsupported sizes give 0
    assert L.vfa_paged_decode_split_workspace_bytes(4, 32, 8, 96, 4) == 0       # head_dim
    assert L.vfa_paged_decode_split_workspace_bytes(4, 30, 8, 128, 4) == 0      # Hq % Hkv
    assert L.vfa_paged_decode_split_workspace_bytes(4, 32, 8, 128, 0) == 0      # runs
    assert L.vfa_paged_decode_split_workspace_bytes(4, 32, 8, 128, 1025) == 0
    assert L.vfa_paged_decode_split_workspace_bytes(0, 32, 8, 128, 4) == 0
    # run count: null result pointer and bad sizes
    n = ctypes.c_int(0)
    assert L.vfa_paged_decode_split_count(4, 8, 32, None) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_paged_decode_split_count(0, 8, 32, ctypes.byref(n)) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_paged_decode_split_count(4, 0, 32, ctypes.byref(n)) == vfa.VFA_ERR_INVALID_ARG
    # split step: run count outside [1, 1024], missing or misaligned workspace,
    # too small a workspace
    fake = ctypes.c_void_p(0x100000)
    ws = ctypes.c_void_p(0x200000)
    step = lambda splits, w, wbytes: L.vfa_paged_decode_step_split(
        fake, fake, fake, 64, fake, fake, None, 32, 4, 32, 8, 128, 16, 0.1, fake, fake, fake,
        None, splits, w, wbytes, None)
    assert step(0, ws, 1 << 30) == vfa.VFA_ERR_INVALID_ARG
    assert step(1025, ws, 1 << 30) == vfa.VFA_ERR_INVALID_ARG
    assert b"num_splits" in L.vfa_last_error()
    assert step(4, None, 1 << 30) == vfa.VFA_ERR_INVALID_ARG
    assert step(4, ctypes.c_void_p(0x200010), 1 << 30) == vfa.VFA_ERR_INVALID_ARG
    need = L.vfa_paged_decode_split_workspace_bytes(4, 32, 8, 128, 4)
    assert step(4, ws, need - 1) == vfa.VFA_ERR_INVALID_ARG
    assert b"too small" in L.vfa_last_error()


def test_norm_rotation_host_checks(vfa):
    L = vfa.lib()
    f = ctypes.c_void_p(0x100000)              # never dereferenced
    odd = ctypes.c_void_p(0x100008)

    def fwd(q=f, stride=512, pos=f, axes=1, table=f, rot=64, eps=1e-6, T=4, Hq=4, Hkv=2, D=128,
            out=f):
        return L.vfa_qk_norm_rope_fwd(q, f, stride, 256, pos, axes, table, rot, 0, f, f, eps, T,
                                      Hq, Hkv, D, out, f, 512, 256, None)

    assert fwd(D=96, stride=1024) == vfa.VFA_ERR_UNSUPPORTED
    assert fwd(Hq=65536, stride=1 << 30) == vfa.VFA_ERR_UNSUPPORTED
    assert fwd(rot=24) == vfa.VFA_ERR_UNSUPPORTED and b"rotary_dim" in L.vfa_last_error()
    for kw in (dict(q=None), dict(out=None), dict(q=odd), dict(stride=508), dict(stride=504),
               dict(pos=None), dict(table=None), dict(table=odd), dict(axes=0), dict(rot=144),
               dict(rot=-16), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(T=-1), dict(Hq=0)):
        assert fwd(**kw) == vfa.VFA_ERR_INVALID_ARG, kw
    assert L.vfa_qk_norm_rope_bwd_workspace_bytes(96) == 0
    need = L.vfa_qk_norm_rope_bwd_workspace_bytes(128)
    assert need > 0

    def bwd(qw=f, dqw=f, ws=f, n=need, dy=f):
        return L.vfa_qk_norm_rope_bwd(f, f, 512, 256, dy, f, 512, 256, f, 1, f, 64, 0, qw, None,
                                      1e-6, 4, 4, 2, 128, f, f, 512, 256, dqw, None, ws, n, None)

    for kw in (dict(dqw=None), dict(ws=None), dict(ws=odd), dict(n=need - 1), dict(dy=None)):
        assert bwd(**kw) == vfa.VFA_ERR_INVALID_ARG, kw


def test_kv4_host_checks(vfa):
    L = vfa.lib()
    f, odd = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008)
    assert L.vfa_kv4_block_bytes(8, 128) == 8 * 18 * 128
    assert L.vfa_kv4_block_bytes(8, 96) == 0 and L.vfa_kv4_block_bytes(0, 128) == 0

    def write(k=f, stride=256, total=4, pool=f, blocks=9, tables=f, cap=3, cu=f, start=f, S=2,
              D=128, dk=1.0, dv=1.0, fn=L.vfa_kv4_write):
        return fn(k, f, stride, 256, total, pool, blocks, tables, cap, cu, start, S, 2, D, dk, dv,
                  None, None)

    for fn in (L.vfa_kv4_write, L.vfa_kv4_gather):
        assert write(fn=fn, D=96) == vfa.VFA_ERR_UNSUPPORTED
        assert write(fn=fn, blocks=(1 << 26) + 1) == vfa.VFA_ERR_UNSUPPORTED
        assert fn(f, f, 1 << 30, 1 << 30, 4, f, 9, f, 3, f, f, 2, 65536, 128, 1.0, 1.0, None,
                  None) == vfa.VFA_ERR_UNSUPPORTED
        for kw in (dict(k=None), dict(k=odd), dict(pool=None), dict(pool=odd), dict(tables=None),
                   dict(cu=None), dict(start=None), dict(stride=248), dict(stride=257),
                   dict(total=-1), dict(cap=-1), dict(S=0), dict(dk=0.0), dict(dk=3.0),
                   dict(dv=-1.0), dict(dv=float("nan")), dict(dk=float("inf")),
                   dict(dk=2.0 ** -65), dict(dv=2.0 ** 65)):
            assert write(fn=fn, **kw) == vfa.VFA_ERR_INVALID_ARG, kw
    need = L.vfa_kv4_decode_workspace_bytes(4, 32, 8, 128)
    assert need > 0
    assert L.vfa_kv4_decode_workspace_bytes(4, 30, 8, 128) == 0
    assert L.vfa_kv4_decode_workspace_bytes(4, 32, 8, 80) == 0
    assert L.vfa_kv4_decode_workspace_bytes(0, 32, 8, 128) == 0
    ws = ctypes.c_void_p(0x200000)

    def decode(q=f, cap=9, counts=f, S=4, Hq=32, D=128, dk=1.0, scale=0.0, out=f, lse=f, w=ws,
               n=need):
        return L.vfa_kv4_decode(q, f, 64, f, cap, counts, S, Hq, 8, D, dk, 1.0, scale, out, lse,
                                None, w, n, None)

    assert decode(D=96) == vfa.VFA_ERR_UNSUPPORTED
    assert decode(cap=1 << 29, n=1 << 40) == vfa.VFA_ERR_UNSUPPORTED
    # sequences and pages counted together pass 32 bits, although the pages alone do not
    assert decode(S=1 << 22, cap=495, n=1 << 40) == vfa.VFA_ERR_UNSUPPORTED
    assert decode(S=1 << 30, cap=1, n=1 << 40) == vfa.VFA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(q=odd), dict(counts=None), dict(out=None), dict(Hq=30),
               dict(Hq=0), dict(dk=0.3), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(w=None), dict(w=odd), dict(n=need - 1), dict(lse=ctypes.c_void_p(0x100002))):
        assert decode(**kw) == vfa.VFA_ERR_INVALID_ARG, kw


def test_page_operation_host_checks(vfa):
    L = vfa.lib()
    f, odd = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100002)
    need = L.vfa_pages_workspace_bytes(100, 4, 8)
    assert need >= 3 * 100 * 4
    assert L.vfa_pages_workspace_bytes(0, 4, 8) == 0
    assert L.vfa_pages_workspace_bytes((1 << 26) + 1, 4, 8) == 0
    assert L.vfa_pages_workspace_bytes(100, 0, 8) == 0
    assert L.vfa_pages_workspace_bytes(100, 4, -1) == 0
    ptrs = (ctypes.c_void_p * 2)(0x100000, 0x200000)
    sizes = (ctypes.c_int * 2)(64, 128)

    def fork(refs=f, blocks=100, cap=6, S=4, par=f, chi=f, n=8, p=ptrs, sz=sizes, np=2, bs=16,
             ws=f, nb=need):
        return L.vfa_pages_fork(refs, blocks, f, cap, f, S, par, chi, n, p, sz, np, bs, ws, nb,
                                None, None)

    assert fork(blocks=(1 << 26) + 1) == vfa.VFA_ERR_UNSUPPORTED
    assert fork(np=257) == vfa.VFA_ERR_UNSUPPORTED
    bad_ptr = (ctypes.c_void_p * 2)(0x100000, 0x200008)
    null_ptr = (ctypes.c_void_p * 2)(0x100000, None)
    for kw in (dict(refs=None), dict(refs=odd), dict(blocks=0), dict(cap=0), dict(S=0),
               dict(par=None), dict(chi=odd), dict(n=-1), dict(p=None), dict(sz=None),
               dict(np=-1), dict(p=bad_ptr), dict(p=null_ptr),
               dict(sz=(ctypes.c_int * 2)(64, 24)), dict(sz=(ctypes.c_int * 2)(0, 64)),
               dict(bs=0), dict(ws=None), dict(nb=need - 1)):
        assert fork(**kw) == vfa.VFA_ERR_INVALID_ARG, kw
    ext = lambda add=f, ws=f, nb=need: L.vfa_pages_extend(f, 100, f, 6, f, 4, add, 16, ws, nb, None,
                                                          None)
    assert ext(add=None) == vfa.VFA_ERR_INVALID_ARG
    assert ext(ws=odd) == vfa.VFA_ERR_INVALID_ARG
    assert ext(nb=64) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_pages_free(f, 100, f, 6, f, 4, None, 1, 16, None, None) == vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_pages_free(f, 100, f, 6, f, 4, f, -1, 16, None, None) == vfa.VFA_ERR_INVALID_ARG
    comp = lambda ro=f, to=f, nu=f: L.vfa_pages_compact(f, 100, f, 6, f, 4, ptrs, sizes, 2, 16, ro,
                                                        to, nu, f, need, None, None)
    for args in ((None, f, f), (f, None, f), (f, f, None), (odd, f, f)):
        assert comp(*args) == vfa.VFA_ERR_INVALID_ARG
    # empty lists may be NULL: the next check in line is the device's
    none = fork(n=0)
    assert fork(n=0, par=None, chi=None) == none != vfa.VFA_ERR_INVALID_ARG
    assert L.vfa_pages_free(f, 100, f, 6, f, 4, None, 0, 16, None, None) == none
    assert L.vfa_pages_copy(ptrs, sizes, 2, None, None, 0, 9, None, None) == none
    assert fork(n=(1 << 26) + 1, nb=1 << 40) == vfa.VFA_ERR_UNSUPPORTED
    assert L.vfa_pages_workspace_bytes(100, 4, (1 << 26) + 1) == 0
    copy = lambda src=f, n=2, nb=9: L.vfa_pages_copy(ptrs, sizes, 2, src, f, n, nb, None, None)
    assert copy(src=None) == vfa.VFA_ERR_INVALID_ARG
    assert copy(n=-1) == vfa.VFA_ERR_INVALID_ARG and copy(nb=0) == vfa.VFA_ERR_INVALID_ARG


def test_binding_checks_of_the_serving_operators(vfa):
    """Wrong devices, types and shapes are refused before anything is launched."""
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vfa.qk_norm_rope(x, x, i, None)
    with pytest.raises(ValueError, match="CUDA"):
        vfa.kv4_write(x, x, torch.zeros(1, 2, 1152, dtype=torch.uint8), i[None], i, i)
    with pytest.raises(ValueError, match="CUDA"):
        vfa.pages_free(i, i[None], i, i, 16)
    with pytest.raises(ValueError, match="axis per"):
        vfa.rope_table([1.0, 0.5], [0], device="cpu")
    with pytest.raises(ValueError, match="finite"):
        vfa.rope_table([float("nan")], device="cpu")
    with pytest.raises(ValueError, match="axes"):
        vfa.rope_table([1.0], [-1], device="cpu")
    with pytest.raises(vfa.VfaError):
        vfa.alloc_kv4_pool(4, 2, 96, device="cpu")
    assert vfa.alloc_kv4_pool(4, 2, 128, device="cpu").shape == (4, 2, 18 * 128)
    # the table's steps: exact products of position and step stay within 2^-64 turns a position
    import math
    t = vfa.rope_table([1.0, 1e-5, -2.5], [0, 1, 2], device="cpu")
    assert t[:, 1].tolist() == [0, 1, 2]
    for step, f in zip(t[:, 0].tolist(), (1.0, 1e-5, -2.5)):
        turns = (step % 2 ** 64) / 2 ** 64
        assert abs(turns - f / (2 * math.pi) % 1.0) < 1e-15


def test_page_sizes_past_32_bits_are_refused(vfa):
    L = vfa.lib()
    f = ctypes.c_void_p(0x100000)
    ptrs = (ctypes.c_void_p * 1)(0x100000)

    def copy(size):
        return L.vfa_pages_copy(ptrs, (ctypes.c_int * 1)(size), 1, f, f, 2, 9, None, None)

    # past 2^31 - 4096 the 4096-byte pieces of a page are no longer counted in 32 bits
    for size in (2 ** 31 - 16, 2 ** 31 - 4096 + 16):
        assert copy(size) == vfa.VFA_ERR_UNSUPPORTED and b"at most" in L.vfa_last_error()
    need = L.vfa_pages_workspace_bytes(9, 2, 0)
    assert L.vfa_pages_compact(f, 9, f, 3, f, 2, ptrs, (ctypes.c_int * 1)(2 ** 31 - 16), 1, 16, f, f, f,
                               f, need, None, None) == vfa.VFA_ERR_UNSUPPORTED

    class Pool:                                # (a page of more than 4 GiB)
        nbytes = 2 * (2 ** 32 + 16)
        get_device = lambda self: 0
        is_contiguous = lambda self: True
        dim = lambda self: 2
        size = lambda self, i: 2
        data_ptr = lambda self: 0x100000

    with pytest.raises(ValueError, match="32 bits"):
        vfa._pool_list([Pool()], 2, 0)
    with pytest.raises(ValueError, match="32 bits"):
        vfa._fits(5, 2 ** 32 + 16)
    vfa._fits(0, 2 ** 31 - 1)
