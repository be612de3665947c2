"""Edges of the token operators that need no GPU: sizes of empty sides, what the sources of the
kernels must hold, the binding's refusals and the build's parts."""

import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from differentiable_gaussian_splatting_gb300 import build

    build.build()


def _python(code: str, **kw):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300, **kw)


# ---------------------------------------------------------------------------
# sides without tokens
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tq,tk,batch", [(5, 0, 1), (0, 7, 2), (0, 0, 2), (100, 0, 1), (0, 100, 1),
                                         (5000, 0, 1), (0, 5000, 1), (40000, 0, 1), (0, 40000, 3)])
def test_attention_workspace_of_an_empty_side(tq, tk, batch):
    # no pieces: the gradient's two fp32 rows per query, in whole 256 bytes, and the slack.  In a
    # process of its own, since a size that divides by a count of zero ends it.
    heads = [(4, 2, 64), (16, 16, 128), (16, 1, 40)]
    r = _python(f"import differentiable_gaussian_splatting_gb300 as gs\n"
                f"for h in {heads}: print(gs.gs_attention_workspace_bytes({tq}, {tk}, {batch}, *h))")
    assert r.returncode == 0, (r.returncode, r.stderr[-300:])
    assert [int(n) for n in r.stdout.split()] == [(8 * tq * hq + 255) // 256 * 256 + 512
                                                  for hq, _, _ in heads]


@pytest.mark.parametrize("tq,tk", [(5, 0), (40000, 0), (0, 7), (0, 40000)])
def test_attention_calls_with_an_empty_side_check_their_workspace(tq, tk):
    # both calls plan before they compare the workspace's size (status 5: too small)
    r = _python(f"""
import ctypes as C
import differentiable_gaussian_splatting_gb300 as gs
lib, P = gs.library(), 0x100000
h = lambda n: C.byref(gs.Heads(P, n * 64, 64))
s = C.byref(gs.AttentionShape({tq}, {tk}, 1, 4, 2, 64, 0, 0.125))
if {tq}:
    print(lib.gs_attention_fwd(s, h(4), h(2), h(2), None, None, h(4), P, P, 16, None))
print(lib.gs_attention_bwd(s, h(4), h(2), h(2), None, None, h(4), P, h(4), h(4), h(2), h(2), P, 16,
                           None))""")
    assert r.returncode == 0, (r.returncode, r.stderr[-300:])
    assert set(r.stdout.split()) == {"5"}


# ---------------------------------------------------------------------------
# the order of dependent launches
# ---------------------------------------------------------------------------
def _kernels():
    """(file, name, body) of every __global__ function of the library"""
    csrc = os.path.join(ROOT, "differentiable_gaussian_splatting_gb300", "csrc")
    for name in sorted(os.listdir(csrc)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            start = text.index("{", m.end())
            depth, end = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            head = re.sub(r"__launch_bounds__\([^()]*\)", "", text[m.end():start])
            yield name, re.search(r"(\w+)\s*\(", head).group(1), text[start + 1:end - 1]


def test_every_kernel_waits_for_the_one_before_it():
    # All kernels are launched with programmatic serialisation: only griddepcontrol.wait orders a
    # kernel's reads after the writes of those before it, so it comes before anything but
    # declarations, in every block, and no kernel goes without.
    declares = re.compile(r"\s*(extern\s+)?(__shared__|constexpr|using|static_assert)\b")
    seen = []
    for file, name, body in _kernels():
        first = body.split("grid_dep_sync();")[0]
        assert first != body, (file, name, "does not wait")
        left = [x for x in first.split(";") if x.strip() and not declares.match(x)]
        assert not left, (file, name, left)
        seen.append(name)
    assert {"attention_delta_kernel", "attention_fwd_kernel", "attention_join_kernel",
            "attention_sum_kernel", "headnorm_kernel", "dropout_add_kernel"} <= set(seen)


def _source(name):
    path = os.path.join(ROOT, "differentiable_gaussian_splatting_gb300", "csrc", name)
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("file,roles", [("gs_attention_fwd.cu", 1), ("gs_attention_bwd.cu", 2)])
def test_no_copy_or_product_outlives_a_block(file, roles):
    # Whoever issued asynchronous work waits for it last of all, in every case: a producer that
    # has issued its last tile may find that another warp has given up.  (What such a block does
    # cannot be run: here the sources are held to it.)
    text = _source(file)
    guards = re.findall(r"if \(([^{}]*)\) \{([^{}]*)\}", text)
    for condition, body in guards:
        if "drain_ring" in body or "&bar_drain" in body:
            raise AssertionError(("waited for under a condition", condition))
    assert len(re.findall(r"mma_commit\(smem_u32\(&bar_drain\)\);\s*"
                          r"mbar_drain\(smem_u32\(&bar_drain\), 0\);", text)) == roles
    rings = set(re.findall(r"drain_ring<Sh::\w+>\((\w+), \w+\)", text))
    assert rings == ({"bar_full"} if roles == 1 else {"full_q", "full_d", "full_k", "full_v"})
    # tiles that are loaded once, outside the rings
    once = set(re.findall(r"mbar_drain\(smem_u32\(&(bar_[qkvd])\b", text))
    assert once == ({"bar_q"} if roles == 1 else {"bar_q", "bar_k", "bar_v", "bar_d"})


# ---------------------------------------------------------------------------
# the binding, on tensors that have a shape and a CUDA device but no memory
# ---------------------------------------------------------------------------
@pytest.fixture
def fake():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    def make(*shape, dtype=torch.bfloat16):
        with FakeTensorMode():
            return torch.empty(shape, dtype=dtype, device="cuda")

    return make


SLOW_LIBRARY = """
#include <unistd.h>
extern "C" {
int gs_qk_norm_rope(...) { return 0; }
int gs_qk_norm_rope_bwd(...) { return 0; }
int gs_attention_fwd(...) { return 0; }
int gs_attention_bwd(...) { return 0; }
int gs_dropout_add(...) { usleep(500000); return 0; }
int gs_dropout_add_bwd(...) { return 0; }
}
"""

SLOW_CALL = """
import importlib.machinery, importlib.util, threading, time, sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

loader = importlib.machinery.ExtensionFileLoader("gs_token_binding", sys.argv[1])
calls = importlib.util.module_from_spec(importlib.util.spec_from_loader("gs_token_binding", loader))
loader.exec_module(calls)
with FakeTensorMode():
    x = torch.empty(0, device="cuda")
    rng = torch.empty(2, dtype=torch.int64, device="cuda")
calls.dropout_add(x, None, x, rng, 0.1, 0)
stop, ticks = False, []

def tick():
    while not stop:
        ticks.append(time.monotonic())
        time.sleep(0.01)

t = threading.Thread(target=tick)
t.start()
time.sleep(0.05)
a = time.monotonic()
calls.dropout_add(x, None, x, rng, 0.1, 0)
b = time.monotonic()
stop = True
t.join()
print(sum(a < x < b for x in ticks), b - a)
"""


def test_a_call_that_waits_lets_other_threads_run(tmp_path):
    # a launch that waits for room in the queue: here a library whose call takes half a second
    from differentiable_gaussian_splatting_gb300 import build

    (tmp_path / "slow.cpp").write_text(SLOW_LIBRARY)
    subprocess.run(["g++", "-shared", "-fPIC", "-Wl,-soname,libgs.so", "-o",
                    str(tmp_path / "libgs.so"), str(tmp_path / "slow.cpp")], check=True)
    copy = shutil.copy(build.BINDING, tmp_path)
    r = subprocess.run([sys.executable, "-c", SLOW_CALL, copy], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
    ticks, seconds = r.stdout.split()
    assert float(seconds) > 0.4 and int(ticks) >= 5, r.stdout


def test_dropout_arrays_have_one_shape(fake):
    # elements are taken by flat index: another shape would be added in the wrong places
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    f32 = torch.float32
    x, rng = fake(4, 6, dtype=f32), fake(2, dtype=torch.int64)
    for bad in (fake(4, 8, dtype=f32), fake(8, 6, dtype=f32), fake(6, 4, dtype=f32),
                fake(24, dtype=f32), fake(25, dtype=f32), fake(1, 6, dtype=f32)):
        with pytest.raises(ValueError, match="residual"):
            gs.gs_dropout_add(x, bad, x, rng, 0.1, stream=0)
        with pytest.raises(ValueError, match="out"):
            gs.gs_dropout_add(x, None, bad, rng, 0.1, stream=0)
        with pytest.raises(ValueError, match="dx"):
            gs.gs_dropout_add_bwd(x, bad, rng, 0.1, stream=0)
    with pytest.raises(ValueError, match="residual"):
        gs.gs_dropout_add(x, fake(4, 6), x, rng, 0.1, stream=0)


def test_head_norm_weights_are_those_of_one_head(fake):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    x, ws = fake(0, 2, 64), fake(1, dtype=torch.uint8)
    good, bad = fake(64, dtype=torch.float32), fake(2, 64, dtype=torch.float32)
    for name, args in (("q_weight", (bad, None)), ("k_weight", (good, bad))):
        with pytest.raises(ValueError, match=name):
            gs.gs_qk_norm_rope(x, x, *args, None, None, x, x, stream=0)
    for name, args in (("dq_weight", (bad, None)), ("dk_weight", (good, bad))):
        with pytest.raises(ValueError, match=name):
            gs.gs_qk_norm_rope_bwd(x, x, good, good, None, None, x, x, x, x, *args, ws, stream=0)
    gs.gs_qk_norm_rope(x, x, good, good, None, None, x, x, stream=0)  # no tokens: nothing to do


class _NoTruth:
    def __bool__(self):
        raise ZeroDivisionError("no truth value")


def test_conditions_and_streams_that_raise(fake):
    # the caller's own error comes out, and nothing is called with what was left in its place
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    x, ws = fake(0, 2, 64), fake(1, dtype=torch.uint8)
    lse, rng = fake(2, 0, dtype=torch.float32), fake(2, dtype=torch.int64)
    with pytest.raises(ZeroDivisionError):
        gs.gs_qk_norm_rope(x, x, None, None, None, None, x, x, interleaved=_NoTruth(), stream=0)
    with pytest.raises(ZeroDivisionError):
        gs.gs_attention_fwd(x, x, x, x, lse, ws, causal=_NoTruth(), stream=0)
    with pytest.raises(OverflowError):
        gs.gs_dropout_add(x, None, x, rng, 0.1, stream=1 << 80)
    with pytest.raises(TypeError):
        gs.gs_dropout_add(x, None, x, rng, "half", stream=0)
    with pytest.raises(AttributeError):
        gs.gs_dropout_add(x, None, x, rng, 0.1, stream="main")


def test_dimensions_beyond_32_bits(fake):
    # 2^32 + 8 heads are not 8
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    n = 2 ** 32 + 8
    x, wide, long = fake(0, 2, 64), fake(0, n, 64), fake(0, 2, n)
    lse, ws = fake(2, 0, dtype=torch.float32), fake(1, dtype=torch.uint8)
    for a, b in ((wide, x), (x, wide), (long, long)):
        with pytest.raises(ValueError, match="too large"):
            gs.gs_qk_norm_rope(a, b, None, None, None, None, a, b, stream=0)
        with pytest.raises(ValueError, match="too large"):
            gs.gs_attention_fwd(a, b, b, a, lse, ws, stream=0)
    table = fake(4, n, dtype=torch.float32)
    with pytest.raises(ValueError, match="too large"):
        gs.gs_qk_norm_rope(x, x, None, None, table, None, x, x, stream=0)
    cu = fake(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="too large"):
        gs.gs_attention_fwd(x, x, x, x, lse, ws, cu_q=cu, cu_k=cu, stream=0)


# ---------------------------------------------------------------------------
# the build's two parts
# ---------------------------------------------------------------------------
@pytest.fixture
def scratch_build(tmp_path, monkeypatch):
    """The build module with its results in a scratch folder and compilers that write empty
    files: (module, list of what was run, set of what shall fail)"""
    from differentiable_gaussian_splatting_gb300 import build

    ran, fails = [], set()

    def run(cmd, what, verbose):
        if what in fails:
            raise RuntimeError(f"{what} failed")
        ran.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgs.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "gs_token_binding.so"))
    monkeypatch.setattr(build, "_run", run)
    return build, ran, fails


def test_library_builds_without_torch(scratch_build, monkeypatch):
    build, ran, _ = scratch_build
    monkeypatch.setitem(sys.modules, "torch", None)
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "libgs.so" in ran and "token_binding.cpp" not in ran
    assert build.up_to_date()
    with pytest.raises(RuntimeError, match="torch"):
        build.build_binding()


@pytest.mark.parametrize("part", ["token_binding.cpp", "gs_token_binding.so"])
def test_library_builds_beside_a_binding_that_fails(scratch_build, part):
    build, ran, fails = scratch_build
    fails.add(part)
    with pytest.raises(RuntimeError, match=part):
        build.build()
    assert os.path.exists(build.LIB) and build.library_up_to_date()
    assert not os.path.exists(build.BINDING) and not build.up_to_date()
    fails.clear()
    ran.clear()
    build.build()
    assert ran == ["token_binding.cpp", "gs_token_binding.so"] and build.up_to_date()


def test_binding_of_another_torch_is_built_anew(scratch_build, monkeypatch):
    build, ran, _ = scratch_build
    build.build()
    ran.clear()
    build.build()
    assert ran == []
    for name, value in (("torch", "9.9"), ("at", "/elsewhere"), ("changed", 1.0), ("python", ".x")):
        made_for = build._torch_of_binding()
        assert name in made_for
        with monkeypatch.context() as m:
            m.setattr(build, "_torch_of_binding", lambda: {**made_for, name: value})
            assert build.library_up_to_date() and not build.binding_up_to_date()
            ran.clear()
            build.build()
            assert ran == ["token_binding.cpp", "gs_token_binding.so"]
        assert not build.binding_up_to_date()
        build.build()
    os.remove(build.BINDING + ".json")  # from before it was recorded
    assert not build.binding_up_to_date()
