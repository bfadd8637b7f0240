"""The entry points of include/svdq_decoder.h without a GPU: exported symbols, the documented status for
every invalid argument with no HIP call, the binding's buffer checks, and the validation code under
host sanitizers."""
import glob
import os
import re
import shutil
import subprocess

import pytest
import torch

from bit_post_quantized_amd import binding, decoder
from bit_post_quantized_amd import decoder_binding as DB
from tests.test_binding_cpu import Dev, _OTHER

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svdq_decoder.h")
OK, EINVAL, ESHAPE, EALIGN = (binding.SVDQ_OK, binding.SVDQ_EINVAL, binding.SVDQ_ESHAPE,
                              binding.SVDQ_EALIGN)
F, G, ODD = 0x10000, 0x40000, 0x10008   # fake addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run python -m bit_post_quantized_amd.build)")
    return DB.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M)))
    assert set(names) == set(DB.EXPORTED)
    for n in names:
        assert hasattr(lib, n), n
    assert lib.svdq_decoder_version() == 1


def test_norm_validation(lib):
    def call(x=F, xt=0, xs=64, r=F, rt=0, ro=F, g=F, M=2, K=64, eps=1e-6, y=F, q=None, s=None):
        return lib.svdq_rms_norm(x, xt, xs, r, rt, ro, g, M, K, eps, y, q, s, None)

    assert call(M=-1) == EINVAL and call(K=0) == EINVAL and call(K=-8) == EINVAL
    assert call(K=60) == ESHAPE and call(K=(1 << 20) + 8, xs=1 << 21) == ESHAPE and call(M=(1 << 24) + 1) == ESHAPE
    assert call(xs=56) == ESHAPE and call(xs=68) == ESHAPE and call(xs=(1 << 31) + 8) == ESHAPE
    assert call(xt=2) == EINVAL and call(rt=-1) == EINVAL
    assert call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL and call(eps=float("inf")) == EINVAL
    assert call(x=None) == EINVAL and call(y=None) == EINVAL
    assert call(r=None) == EINVAL and b"needs a residual" in lib.svdq_last_error()
    assert call(q=F) == EINVAL and call(s=F) == EINVAL and b"go together" in lib.svdq_last_error()
    for k in ("x", "r", "ro", "g", "y"):
        assert call(**{k: ODD}) == EALIGN, k
    assert call(q=ODD, s=F) == EALIGN
    assert call(M=0) == OK and call(M=0, x=None, r=None, ro=None, y=None) == OK

    def rows(x=F, xt=0, xs=64, f=None, M=2, K=64, q=F, s=F):
        return lib.svdq_quantize_rows(x, xt, xs, f, M, K, q, s, None)

    assert rows(M=-1) == EINVAL and rows(K=12) == ESHAPE and rows(xt=3) == EINVAL and rows(xs=8) == ESHAPE
    assert rows(q=None) == EINVAL and rows(s=None) == EINVAL and rows(x=None) == EINVAL
    assert rows(x=ODD) == EALIGN and rows(f=ODD) == EALIGN and rows(q=ODD) == EALIGN
    assert rows(M=0, x=None, q=None, s=None) == OK


def test_product_validation(lib):
    def call(qx=F, sx=F, w=F, sw=F, b=None, M=2, N=16, K=64, Y=F, out=0, ws=F):
        return lib.svdq_w8a8_gemm(qx, sx, w, sw, b, M, N, K, Y, out, ws, None)

    assert call(M=-1) == EINVAL and call(N=0) == EINVAL and call(K=0) == EINVAL and call(out=2) == EINVAL
    assert call(K=96) == ESHAPE and call(K=64 * 2048) == ESHAPE and call(N=(1 << 24) + 1) == ESHAPE
    assert call(M=(1 << 24) + 1) == ESHAPE and call(M=1 << 24, N=1 << 17) == ESHAPE
    for k in ("qx", "sx", "w", "sw", "Y"):
        assert call(**{k: None}) == EINVAL, k
    for k in ("qx", "w", "Y", "ws"):
        assert call(**{k: ODD}) == EALIGN, k
    assert call(M=200, K=64 * 64, ws=None) == EINVAL and b"workspace" in lib.svdq_last_error()
    assert call(M=0, qx=None, sx=None, Y=None, ws=None) == OK
    w, c, p = lib.svdq_w8a8_workspace_bytes, lib.svdq_w8a8_container_bytes, lib.svdq_pack_w8a8
    assert w(0, 16, 64) == 0 and w(16, 16, 1 << 16) == 0 and w(1, 16, 65) == 0 and w(200, 16, 64 * 64) > 0
    assert c(16, 64) == 1024 and c(17, 128) == 4096 and c(0, 64) == 0 and c(16, 100) == 0 and c(1, 64 * 2048) == 0
    assert p(F, 0, 64, F, None) == EINVAL and p(F, 16, 65, F, None) == ESHAPE and p(None, 16, 64, F, None) == EINVAL
    assert p(F, 16, 64, None, None) == EINVAL and p(ODD, 16, 64, F, None) == EALIGN and p(F, 16, 64, ODD, None) == EALIGN


def test_rope_validation(lib):
    def call(q=F, qs=256, h=4, k=F, ks=128, kv=2, xt=0, rows=3, dim=64, rot=64, pos=F, f=F, scale=1.0, qo=G, qos=256,
             ko=G, kos=128):
        return lib.svdq_rope(q, qs, h, k, ks, kv, xt, rows, dim, rot, 0, pos, f, scale, qo, qos, ko, kos, None)

    assert call(rows=-1) == EINVAL and call(h=0) == EINVAL and call(kv=-1) == EINVAL and call(dim=0) == EINVAL
    assert call(rot=0) == EINVAL and call(rot=24) == ESHAPE and call(rot=80) == ESHAPE and call(dim=60) == ESHAPE
    assert call(dim=1032, qs=1 << 16, ks=1 << 16, qos=1 << 16, kos=1 << 16) == ESHAPE
    assert call(h=65536, qs=1 << 22, qos=1 << 22) == ESHAPE and call(rows=1 << 25) == ESHAPE
    assert call(xt=5) == EINVAL and call(scale=float("nan")) == EINVAL and call(scale=float("inf")) == EINVAL
    for k in ("qs", "qos"):
        assert call(**{k: 248}) == ESHAPE and call(**{k: 260}) == ESHAPE
    for k in ("ks", "kos"):
        assert call(**{k: 120}) == ESHAPE and call(**{k: 132}) == ESHAPE
    for k in ("q", "k", "pos", "f", "qo", "ko"):
        assert call(**{k: None}) == EINVAL, k
    for k in ("q", "k", "f", "qo", "ko"):
        assert call(**{k: ODD}) == EALIGN, k
    # in place: bf16 and the same rows only
    assert call(qo=F, xt=1) == EINVAL and call(qo=F, qos=264) == EINVAL and call(ko=F, kos=136) == EINVAL
    assert call(rows=0, q=None, k=None, pos=None, qo=None, ko=None) == OK and call(rows=0, kv=0, k=None, ko=None) == OK


def test_sample_validation(lib):
    def call(z=F, zt=0, zs=100, rows=2, vocab=100, t=F, u=F, tokens=F, ws=F):
        return lib.svdq_sample(z, zt, zs, rows, vocab, t, u, None, None, None, tokens, None, ws, None)

    assert call(rows=-1) == EINVAL and call(vocab=0) == EINVAL and call(zt=2) == EINVAL
    assert call(rows=65536) == ESHAPE and call(vocab=(1 << 22) + 1, zs=1 << 23) == ESHAPE
    assert call(zs=99) == ESHAPE and call(zs=(1 << 31) + 1) == ESHAPE
    for k in ("z", "t", "u", "tokens", "ws"):
        assert call(**{k: None}) == EINVAL, k
    assert call(ws=ODD) == EALIGN and call(z=F + 1) == EALIGN and call(z=F + 2, zt=1) == EALIGN
    assert call(rows=0, z=None, t=None, u=None, tokens=None, ws=None) == OK
    w = lib.svdq_sample_workspace_bytes
    assert w(0, 100) == 0 and w(1, 0) == 0 and w(65536, 100) == 0 and w(2, 100) > 0
    # a row's list has 32 KiB, each of at most 1024 chunks (4096 where rows are done in batches) under 20 KiB of bins
    # and maxima
    assert w(64, 131072) <= 64 * (33 << 10) + 1024 * (20 << 10)
    assert w(65535, 1 << 22) <= 4096 * (33 << 10) + 4096 * (20 << 10) and w(65535, 1) == w(4096, 1)


def _cases():
    bf16, f32, f64, i8, i32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32
    M, K, N, V = 200, 64 * 64, 40, 300
    return [
        (DB.svdq_rms_norm, ["x", "residual", "residual_out", "gamma", "eps", "y", "codes", "scales"],
         dict(residual=([M, K], bf16), residual_out=([M, K], bf16), gamma=([K], f32), y=([M, K], bf16),
              codes=([M, K], i8), scales=([M], f32)), dict(eps=1e-6), dict(x=([M, K], bf16))),
        (DB.svdq_quantize_rows, ["x", "factor", "codes", "scales"],
         dict(factor=([K], f32), codes=([M, K], i8), scales=([M], f32)), {}, dict(x=([M, K], bf16))),
        (DB.svdq_pack_w8a8, ["codes", "container"],
         dict(codes=([N, K], i8), container=([DB.svdq_w8a8_container_bytes(N, K)], i8)), {}, {}),
        (DB.svdq_w8a8_gemm, ["qx", "sx", "container", "sw", "bias", "Y", "workspace"],
         dict(qx=([M, K], i8), sx=([M], f32), container=([DB.svdq_w8a8_container_bytes(N, K)], i8), sw=([N], f32),
              bias=([N], bf16), Y=([M, N], bf16), workspace=([DB.svdq_w8a8_workspace_bytes(M, N, K)], torch.uint8)), {}, {}),
        (DB.svdq_sample, ["logits", "temperature", "uniform", "top_k", "top_p", "min_p", "tokens", "share", "workspace"],
         dict(temperature=([M], f32), uniform=([M], f32), top_k=([M], i32), top_p=([M], f32), min_p=([M], f32),
              tokens=([M], i32), share=([M], f32), workspace=([DB.svdq_sample_workspace_bytes(M, V)], torch.uint8)), {},
         dict(logits=([M, V], f32))),
        (DB.svdq_rope, ["q", "k", "positions", "freqs", "interleaved", "scale", "q_out", "k_out"],
         dict(positions=([M], i32), freqs=([32], f64)), dict(interleaved=False, scale=1.0),
         dict(q=([M, 4, 64], bf16), k=([M, 2, 64], bf16), q_out=([M, 4, 64], bf16), k_out=([M, 2, 64], bf16))),
    ]


OTHER = dict(_OTHER)
OTHER.update({torch.int8: torch.uint8, torch.float64: torch.int64, torch.int32: torch.float32})


class Rows(Dev):
    """A fake device tensor whose rows stand next to each other."""

    def __init__(self, shape, dtype):
        super().__init__(shape, dtype)
        self._strides = []
        size = 1
        for n in reversed(shape):
            self._strides.insert(0, size)
            size *= n

    def stride(self, i=None):
        return tuple(self._strides) if i is None else self._strides[i]


@pytest.mark.parametrize("case", _cases(), ids=lambda c: c[0].__name__)
def test_short_buffers_and_wrong_dtypes_are_rejected_by_name(lib, case):
    fn, order, tensors, scalars, strided = case
    for name in tensors:
        given = lambda k: scalars[k] if k in scalars else Rows(*strided[k])  # noqa: E731
        args = [given(k) if k not in tensors else Dev(*tensors[k], short=(k == name)) for k in order]
        with pytest.raises(ValueError, match=f"{fn.__name__}: {name} holds .* bytes"):
            fn(*args)
        if name == "workspace":
            continue
        args = [given(k) if k not in tensors else
                Dev(*tensors[k], as_dtype=OTHER[tensors[k][1]] if k == name else None) for k in order]
        want = f"{name} must be" if name in ("Y", "residual") else f"{name} must be {tensors[name][1]}"
        with pytest.raises(ValueError, match=re.escape(f"{fn.__name__}: {want}")):
            fn(*args)


def test_wrong_shapes_are_refused(lib):
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k = Rows([3, 4, 64], bf16), Rows([3, 2, 64], bf16)
    pos, freqs = Dev([3], i32), Dev([32], torch.float64)
    with pytest.raises(ValueError, match="same dtype"):
        DB.svdq_rope(q, Rows([3, 2, 64], f32), pos, freqs, False, 1.0, q, k)
    with pytest.raises(ValueError, match="same rows"):
        DB.svdq_rope(q, Rows([4, 2, 64], bf16), pos, freqs, False, 1.0, q, Rows([4, 2, 64], bf16))
    with pytest.raises(ValueError, match="k needs k_out"):
        DB.svdq_rope(q, k, pos, freqs, False, 1.0, q, None)
    with pytest.raises(ValueError, match="q_out must have 3 rows"):
        DB.svdq_rope(q, k, pos, freqs, False, 1.0, Rows([5, 4, 64], bf16), k)
    with pytest.raises(ValueError, match="k_out must be"):
        DB.svdq_rope(q, k, pos, freqs, False, 1.0, q, Rows([3, 2, 64], f32))
    with pytest.raises(ValueError, match="contiguous rows"):
        DB.svdq_rope(q, Rows([3, 2, 128], bf16), pos, freqs, False, 1.0, q, k)
    with pytest.raises(ValueError, match="x must be bfloat16 or float32"):
        DB.svdq_quantize_rows(Rows([3, 64], torch.float16), None, Dev([3, 64], torch.int8), Dev([3], f32))


def test_host_tensors_are_rejected(lib):
    x, s = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3)
    with pytest.raises(ValueError, match="device tensor"):
        decoder.RMSNorm(torch.ones(64))
    with pytest.raises(ValueError, match="device tensor"):
        decoder.quantize_rows(x)
    with pytest.raises(ValueError, match="device tensor"):
        decoder.Linear8(torch.zeros(16, 64, dtype=torch.int8), torch.zeros(16))
    with pytest.raises(ValueError, match="device tensor"):
        decoder.Rope(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="device tensor"):
        decoder.sample(x.float(), s, s)


def test_validation_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    """abi.cpp and abi_decoder.cpp built for the host with the sanitizers, and a driver that calls the
    entry points with extreme arguments; nothing reaches a launch."""
    from bit_post_quantized_amd import build

    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    objs = sorted(o for o in glob.glob(os.path.join(build.OBJDIR, "*.o"))
                  if os.path.basename(o) not in ("abi.o", "abi_decoder.o", "peaks.o"))
    if not objs:
        pytest.fail("kernel objects are not built (run python -m bit_post_quantized_amd.build)")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    sanitize = ["-fsanitize=" + "address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    common = ["-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
              f"-I{os.path.join(ROOT, 'include')}", f"-I{build.CSRC}", *sanitize]
    made = []
    for src in (os.path.join(build.CSRC, "abi.cpp"), os.path.join(build.CSRC, "abi_decoder.cpp"),
                os.path.join(ROOT, "tests", "decoder_sanitize_main.cpp")):
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
