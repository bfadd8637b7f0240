"""The decoding step's entry points (include/svdq_serve.h) without a GPU: exported symbols, the
documented status for every invalid argument with no HIP call, the binding's buffer checks, and
the validation code under host sanitizers."""
import glob
import os
import re
import shutil
import subprocess

import pytest
import torch

from bit_post_quantized_amd import binding, layer, serve
from bit_post_quantized_amd import serve_binding as SB
from tests.test_binding_cpu import Dev, _OTHER

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svdq_serve.h")
OK, EINVAL, ESHAPE, EALIGN = (binding.SVDQ_OK, binding.SVDQ_EINVAL, binding.SVDQ_ESHAPE,
                              binding.SVDQ_EALIGN)
F, ODD = 0x10000, 0x10008   # fake addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run python -m bit_post_quantized_amd.build)")
    return SB.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M)))
    assert set(names) == set(SB.EXPORTED)
    for n in names:
        assert hasattr(lib, n), n
    assert lib.svdq_serve_version() == 1


def test_gemv_validation(lib):
    f = lib.svdq_w4a16_gemv

    def call(M=1, N=16, K=64, r=0, X=F, inv=F, l1=F, wt=F, l2=F, bias=None, Y=F, out=0, wsp=F):
        return f(X, inv, l1, wt, l2, bias, M, N, K, r, Y, out, wsp, None)

    assert call(M=-1) == EINVAL and call(N=0) == EINVAL and call(K=0) == EINVAL and call(r=-16) == EINVAL
    assert call(K=100) == ESHAPE and call(r=24) == ESHAPE and call(r=144) == ESHAPE
    assert call(M=65) == ESHAPE and b"svdq_w4a4_gemm" in lib.svdq_last_error()
    assert call(N=(1 << 24) + 1) == ESHAPE and call(K=64 * 65536) == ESHAPE
    assert call(N=1 << 24, K=64 * 65535) == ESHAPE      # N K past 2^40
    assert call(out=2) == EINVAL
    assert call(X=None) == EINVAL and call(Y=None) == EINVAL and call(wsp=None) == EINVAL and call(wt=None) == EINVAL
    assert call(r=16, l1=None) == EINVAL and call(r=16, l2=None) == EINVAL
    for k in ("X", "inv", "wt", "wsp"):
        assert call(**{k: ODD}) == EALIGN
    assert call(r=16, l1=ODD) == EALIGN and call(r=16, l2=ODD) == EALIGN
    assert call(M=0) == OK and call(M=0, X=None, Y=None, wsp=None) == OK
    w = lib.svdq_w4a16_workspace_bytes
    assert w(0, 16, 64, 0, 0) == 0 and w(65, 16, 64, 0, 0) == 0 and w(1, 16, 100, 0, 0) == 0
    # one row tile of 16 rows x 64 k of fp16, its 16 scales, and T's partials
    assert w(1, 16, 64, 16, 0) == 2048 + 64 + 16 * 4
    assert w(9, 16, 128, 0, 1) == 2 * (2 * 2048 + 64)   # fp32 output: 8 rows to a tile
    p, c = lib.svdq_pack_w4a16, lib.svdq_w4a16_container_bytes
    assert p(F, F, 0, 64, F, None) == EINVAL and p(F, F, 16, 65, F, None) == ESHAPE
    assert p(None, F, 16, 64, F, None) == EINVAL and p(F, F, 16, 64, None, None) == EINVAL
    assert p(ODD, F, 16, 64, F, None) == EALIGN and p(F, F, 16, 64, ODD, None) == EALIGN
    assert c(16, 512) == 4352 and c(17, 576) == 4 * 4352 and c(0, 512) == 0 and c(16, 100) == 0
    assert c(1 << 24, 64 * 65535) == 0


def test_plan_and_release_validation(lib):
    p = lib.kv_block_plan

    def plan(n=2, width=4, bs=16, cap=8, rows=4, count=F, out=0x20000, ptr=F):
        return p(ptr, ptr, n, ptr, width, bs, ptr, cap, count, ptr, ptr, rows, ptr, ptr, ptr, out, None)

    assert plan(n=-1) == EINVAL and plan(width=0) == EINVAL and plan(rows=-1) == EINVAL and plan(cap=-1) == EINVAL
    assert plan(bs=8) == ESHAPE and plan(bs=48) == ESHAPE and plan(bs=256) == ESHAPE
    assert plan(n=(1 << 20) + 1) == ESHAPE and plan(n=1 << 20, width=2048) == ESHAPE
    assert plan(n=1, width=1 << 27) == ESHAPE and plan(rows=(1 << 30) + 1) == ESHAPE
    assert plan(ptr=None) == EINVAL and plan(count=None) == EINVAL and plan(out=None) == EINVAL
    assert plan(out=F) == EINVAL and b"free_count_out" in lib.svdq_last_error()
    r = lib.kv_block_release
    assert r(F, F, -1, F, 4, 16, F, 8, F, 0x20000, 0x20000, None) == EINVAL
    assert r(F, F, 2, F, 4, 20, F, 8, F, 0x20000, 0x30000, None) == ESHAPE
    assert r(F, F, 2, F, 4, 16, F, 8, F, F, 0x30000, None) == EINVAL
    assert r(F, F, 2, F, 4, 16, F, 8, F, 0x20000, F, None) == EINVAL
    assert r(F, None, 2, F, 4, 16, F, 8, F, 0x20000, 0x30000, None) == EINVAL


def test_append_and_read_validation(lib):
    def append(k=F, v=F, ks=256, vs=256, slots=F, rows=1, heads=2, dim=64, bs=16, num=4, kc=F, vc=F, s=F):
        return lib.kv_block_append(k, v, ks, vs, slots, rows, heads, dim, bs, num, kc, vc, s, s, None)

    assert append(rows=-1) == EINVAL and append(heads=0) == EINVAL and append(num=0) == EINVAL
    assert append(dim=96) == ESHAPE and append(bs=24) == ESHAPE and append(heads=65536) == ESHAPE
    assert append(num=2 ** 31 - 1, heads=65535, ks=1 << 24, vs=1 << 24) == ESHAPE
    assert append(ks=127) == ESHAPE and append(vs=129) == ESHAPE and append(ks=120) == ESHAPE
    assert append(rows=(1 << 30) + 1) == ESHAPE
    assert append(rows=(1 << 26) + 1) == ESHAPE and b"rows * kv_heads" in lib.svdq_last_error()
    for k in ("k", "v", "slots", "kc", "vc", "s"):
        assert append(**{k: None}) == EINVAL, k
    for k in ("k", "v", "kc", "vc"):
        assert append(**{k: ODD}) == EALIGN, k
    assert append(rows=0, k=None, v=None, slots=None) == OK

    def read(slots=F, rows=1, heads=2, dim=64, bs=16, num=4, kc=F, vc=F, s=F, ko=F, vo=F):
        return lib.kv_block_read(slots, rows, heads, dim, bs, num, kc, vc, s, s, ko, vo, None)

    assert read(rows=(1 << 26) + 1) == ESHAPE and b"rows * kv_heads" in lib.svdq_last_error()
    assert read(rows=-1) == EINVAL and read(dim=32) == ESHAPE and read(bs=1) == ESHAPE
    for k in ("slots", "kc", "vc", "s", "ko", "vo"):
        assert read(**{k: None}) == EINVAL, k
    for k in ("kc", "vc", "ko", "vo"):
        assert read(**{k: ODD}) == EALIGN, k
    assert read(rows=0, slots=None, ko=None, vo=None) == OK


def test_attention_validation(lib):
    def call(q=F, qs=512, kc=F, vc=F, s=F, tables=F, width=4, seq=F, cu=F, n=2, rows=2, most=1, heads=8,
             kv=2, dim=64, bs=16, num=9, causal=1, sm=0.125, out=F, wsp=F):
        return lib.kv_block_attention(q, qs, kc, vc, s, s, tables, width, seq, cu, n, rows, most, heads,
                                      kv, dim, bs, num, causal, sm, out, wsp, None)

    assert call(n=-1) == EINVAL and call(rows=-1) == EINVAL and call(most=0) == EINVAL
    assert call(heads=0) == EINVAL and call(kv=0) == EINVAL and call(width=0) == EINVAL and call(num=0) == EINVAL
    assert call(heads=7) == ESHAPE and call(heads=258) == ESHAPE and call(dim=80) == ESHAPE and call(bs=12) == ESHAPE
    assert call(n=65536) == ESHAPE and call(rows=(1 << 24) + 1) == ESHAPE and call(most=(1 << 24) + 1) == ESHAPE
    assert call(n=65535, heads=129, kv=129, qs=129 * 64, rows=1 << 24) == ESHAPE  # 2^23 workgroups
    assert b"too many rows" in lib.svdq_last_error()
    assert call(n=60000, rows=1 << 24, most=1 << 24) == ESHAPE and b"too many rows" in lib.svdq_last_error()
    assert call(qs=504) == ESHAPE and call(qs=513) == ESHAPE
    assert call(sm=float("nan")) == EINVAL and call(sm=float("inf")) == EINVAL
    for k in ("q", "kc", "vc", "s", "tables", "seq", "cu", "out"):
        assert call(**{k: None}) == EINVAL, k
    for k in ("q", "kc", "vc", "out", "wsp"):
        assert call(**{k: ODD}) == EALIGN, k
    assert call(wsp=None, width=4096) == EINVAL and b"workspace" in lib.svdq_last_error()
    assert call(n=0) == OK and call(rows=0, q=None, out=None) == OK
    w = lib.kv_block_attention_workspace_bytes
    assert w(0, 0, 1, 8, 2, 64, 4, 16) == 0 and w(2, 2, 1, 7, 2, 64, 4, 16) == 0
    assert w(1, 1, 1, 8, 2, 64, 1, 16) == 0         # a short table is not split
    assert w(1, 1, 1, 8, 2, 64, 65536, 16) > 0


def _cases():
    bf16, f16, f32, u8, i32, i64 = (torch.bfloat16, torch.float16, torch.float32, torch.uint8,
                                    torch.int32, torch.int64)
    M, K, N, R = 3, 192, 40, 16
    num, H, bs, D, n, width, rows = 5, 2, 16, 64, 3, 4, 7
    cache = dict(k_codes=([num, H, bs, D], u8), v_codes=([num, H, D, bs], u8), k_scale=([num, H], f32),
                 v_scale=([num, H], f32))
    names = list(cache)
    plan = dict(block_tables=([n, width], i32), free_blocks=([9], i32), free_count=([1], i32))
    return [
        (SB.svdq_pack_w4a16, ["wq", "w_scales", "container"],
         dict(wq=([N, K // 2], u8), w_scales=([K // 64, N], f16),
              container=([SB.svdq_w4a16_container_bytes(N, K)], u8)), {}),
        (SB.svdq_w4a16_gemv, ["X", "inv_lambda", "L1p", "container", "L2p", "bias", "r", "Y", "workspace"],
         dict(X=([M, K], bf16), inv_lambda=([K], f32), L1p=([R, K], bf16),
              container=([SB.svdq_w4a16_container_bytes(N, K)], u8), L2p=([N, R], bf16), bias=([N], bf16),
              Y=([M, N], bf16), workspace=([SB.svdq_w4a16_workspace_bytes(M, N, K, R, 0)], u8)), dict(r=R)),
        (SB.kv_block_plan, ["ctx_lens", "new_lens", "block_tables", "block_size", "free_blocks", "free_count",
                            "cu_rows", "seq_lens", "positions", "slots", "status", "free_count_out"],
         dict(plan, ctx_lens=([n], i32), new_lens=([n], i32), cu_rows=([n + 1], i32), seq_lens=([n], i32),
              positions=([rows], i32), slots=([rows], i64), status=([n], i32), free_count_out=([1], i32)),
         dict(block_size=bs)),
        (SB.kv_block_release, ["seq_lens", "done", "block_tables", "block_size", "free_blocks", "free_count",
                               "seq_lens_out", "free_count_out"],
         dict(plan, seq_lens=([n], i32), done=([n], u8), seq_lens_out=([n], i32), free_count_out=([1], i32)),
         dict(block_size=bs)),
        (SB.kv_block_read, ["slots", *names, "k_out", "v_out"],
         dict(cache, slots=([rows], i64), k_out=([rows, H, D], bf16), v_out=([rows, H, D], bf16)), {}),
    ]


OTHER = dict(_OTHER)
OTHER[torch.int64] = torch.float64


@pytest.mark.parametrize("case", _cases(), ids=lambda c: c[0].__name__)
def test_short_buffers_and_wrong_dtypes_are_rejected_by_name(lib, case):
    fn, order, tensors, scalars = case
    for name in tensors:
        args = [scalars[k] if k in scalars else Dev(*tensors[k], short=(k == name)) for k in order]
        with pytest.raises(ValueError, match=f"{fn.__name__}: {name} holds .* bytes"):
            fn(*args)
        if name == "workspace":
            continue
        args = [scalars[k] if k in scalars else
                Dev(*tensors[k], as_dtype=OTHER[tensors[k][1]] if k == name else None) for k in order]
        want = "Y must be" if name == "Y" else f"{name} must be {tensors[name][1]}"
        with pytest.raises(ValueError, match=re.escape(f"{fn.__name__}: {want}")):
            fn(*args)


def test_host_tensors_are_rejected(lib):
    cache = [torch.zeros(5, 2, 16, 64, dtype=torch.uint8), torch.zeros(5, 2, 64, 16, dtype=torch.uint8),
             torch.zeros(5, 2), torch.zeros(5, 2)]
    x, s = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        serve.BlockCache(*cache)
    with pytest.raises(ValueError, match="device tensor"):
        SB.kv_block_append(x, x, s, *cache)
    with pytest.raises(ValueError, match="device tensor"):
        SB.kv_block_read(s, *cache, x, x)
    with pytest.raises(ValueError, match="device tensor"):
        SB.kv_block_attention(x, *cache, i[None], i, torch.zeros(2, dtype=torch.int32), 1, True, 1.0, x, None)
    with pytest.raises(ValueError, match="device tensor"):
        serve.BlockPlanner(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 16, 4)


def test_the_tiled_container_is_refused():
    pw = layer.PackedWeights(K=64, N=16, rank=0, inv_lambda=None, L1p=None, L2p=None, wq=None,
                             w_scales=None, e3m2=True)
    with pytest.raises(ValueError, match="nibble container"):
        serve.DecodeLinear(pw)


def test_validation_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    """abi.cpp and abi_serve.cpp built for the host with the sanitizers, and a driver that calls
    the decoding step's entry points with extreme arguments; nothing reaches a launch."""
    from bit_post_quantized_amd import build

    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    objs = sorted(o for o in glob.glob(os.path.join(build.OBJDIR, "*.o"))
                  if os.path.basename(o) not in ("abi.o", "abi_serve.o", "peaks.o"))
    if not objs:
        pytest.fail("kernel objects are not built (run python -m bit_post_quantized_amd.build)")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    sanitize = ["-fsanitize=" + "address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    common = ["-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
              f"-I{os.path.join(ROOT, 'include')}", f"-I{build.CSRC}", *sanitize]
    made = []
    for src in (os.path.join(build.CSRC, "abi.cpp"), os.path.join(build.CSRC, "abi_serve.cpp"),
                os.path.join(ROOT, "tests", "serve_sanitize_main.cpp")):
        made.append(str(tmp_path / (os.path.basename(src) + ".o")))
        res = subprocess.run([gxx, *common, "-c", src, "-o", made[-1]], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-3000:]
    exe = str(tmp_path / "check")
    res = subprocess.run([gxx, *sanitize, *made, *objs, f"-L{rocm}/lib", "-lamdhip64",
                          f"-Wl,-rpath,{rocm}/lib", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    report = run.stdout + run.stderr
    assert run.returncode == 0 and "runtime error" not in report and "AddressSanitizer" not in report, report[-3000:]
    assert "all checks passed" in run.stdout
