"""The layer operators without a GPU: the oracle's gradients against differences and closed forms, the C ABI's
layout and exports, and every refusal that needs no device."""

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from persistent_tiled_gemm_amd import layer

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ptg_layer.h")
INVALID, SHAPE = -1, -2


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("name", ref.ACTIVATIONS)
def test_oracle_activation_gradient_is_its_difference(name):
    z = torch.linspace(-6, 6, 1001, dtype=torch.float64)
    z = z[z.abs() > 1e-3]
    h = 1e-5
    diff = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    assert (diff - ref.act_grad(z, name)).abs().max() < 1e-8


def test_oracle_activation_values():
    one = torch.ones(1, dtype=torch.float64)
    assert abs(ref.act(one, "gelu").item() - 0.8413447460685429) < 1e-15   # Phi(1)
    assert abs(ref.act(one, "silu").item() - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(ref.act(one, "gelu_tanh").item() - 0.8411919906082768) < 1e-12
    assert ref.act(-one, "relu").item() == 0.0


def test_oracle_norm_gradient_is_its_difference():
    x, w, dy = rand(5, 24, seed=1), rand(24, seed=2), rand(5, 24, seed=3)
    dx, dw = ref.rmsnorm_backward(dy, x, w)
    h = 1e-6
    for seed in range(4):
        u, v = rand(5, 24, seed=10 + seed), rand(24, seed=20 + seed)
        loss = lambda t: (ref.rmsnorm(x + t * u, w + t * v)[1] * dy).sum()  # noqa: E731
        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - ((dx * u).sum() + (dw * v).sum())) < 1e-7


def test_oracle_quantise():
    y = torch.tensor([[0.0, 0.0], [1.0, -2.0], [448.0, 7.0]], dtype=torch.float64)
    scale, v = ref.quantise(y)
    assert scale.tolist() == [1.0, 2.0 / 448.0, 1.0]
    assert v.abs().amax(dim=1).tolist() == [0.0, 448.0, 448.0]


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(layer_[a-z_0-9]+)\s*\(", text, flags=re.M)))


def test_header_binding_and_library_name_the_same_functions():
    assert declared() == sorted(ptg.LAYER_ABI_FUNCTIONS)
    out = subprocess.run(["nm", "-D", "--defined-only", ptg.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(declared()) <= set(re.findall(r"\sT\s(layer_[a-z_0-9]+)$", out, flags=re.M))


def test_struct_layouts_match_the_binding(tmp_path):
    structs = {"layer_rmsnorm_args": layer.RmsnormArgs, "layer_rmsnorm_grad_args": layer.RmsnormGradArgs,
               "layer_linear_args": layer.LinearArgs, "layer_activation_grad_args": layer.ActivationGradArgs,
               "layer_linear_grad_args": layer.LinearGradArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "ptg_layer.h"', "int main(void) {"]
    for c, cls in structs.items():
        lines.append(f'  printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'  printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = dict(x.rsplit(" ", 1) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, cls in structs.items():
        assert int(got[c]) == ctypes.sizeof(cls), c
        for f, _ in cls._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(cls, f).offset, (c, f)


# ---- refusals: none of these calls reaches the device. Pointers are made up and never followed.

P = 0x100000


def call_rmsnorm(**kw):
    a = layer.RmsnormArgs(x=P, weight=P, out=P, m=4, n=64, ldx=64, ldr=64, lds=64, ldo=64, type=1, weight_type=1, out_type=1, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return layer._library().layer_rmsnorm(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=7), INVALID), (dict(out_type=3), INVALID), (dict(weight_type=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(out=P + 8), INVALID), (dict(residual=P + 4), INVALID), (dict(sum_out=P + 4), INVALID),
    (dict(weight=P + 2), INVALID), (dict(out_type=2), INVALID), (dict(scale=P), INVALID), (dict(out_type=2, scale=P + 2), INVALID),
    (dict(n=63), SHAPE), (dict(n=-8), SHAPE), (dict(m=-1), SHAPE), (dict(n=(1 << 15) + 8, ldx=1 << 16, ldo=1 << 16), SHAPE),
    (dict(ldx=56), SHAPE), (dict(ldo=68), SHAPE), (dict(residual=P, ldr=8), SHAPE), (dict(sum_out=P, lds=8), SHAPE),
    (dict(m=(1 << 30) + 1), SHAPE), (dict(ldx=(1 << 20) + 8), SHAPE)])
def test_rmsnorm_refuses(kw, status):
    assert call_rmsnorm(**kw) == status


def test_empty_rmsnorm_is_accepted_without_a_device():
    assert call_rmsnorm(m=0, x=None, out=None) == 0
    assert call_rmsnorm(n=0, x=None, out=None) == 0
    assert call_rmsnorm(m=0, x=None, out=None, out_type=2) == 0


def test_null_structs_and_plans_are_refused():
    lib = layer._library()
    assert lib.layer_rmsnorm(None, None) == INVALID
    assert lib.layer_create(None, 0) == INVALID
    assert lib.layer_sync(None) == INVALID
    assert lib.layer_destroy(None) == 0
    assert lib.layer_last_hip_error(None) == b""
    for f, cls in ((lib.layer_rmsnorm_backward, layer.RmsnormGradArgs), (lib.layer_linear, layer.LinearArgs),
                   (lib.layer_activation_backward, layer.ActivationGradArgs), (lib.layer_linear_backward, layer.LinearGradArgs)):
        assert f(None, None, None) == INVALID
        assert f(ctypes.byref(cls()), None, None) == INVALID  # no plan


def test_binding_refuses_host_tensors_and_bad_names():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ptg.layer_rmsnorm(x, None, x)
    with pytest.raises(ValueError):
        ptg.layer_rmsnorm(x[0], None, x)

    class Plan:
        handle, device = None, 0
    with pytest.raises(ValueError):
        ptg.layer_linear(x, x, x, Plan(), activation="tanh")
    with pytest.raises(ValueError):
        ptg.layer_linear(x, torch.zeros(8, 16, dtype=torch.bfloat16), x, Plan())
    with pytest.raises(ValueError):
        ptg.layer_linear_backward(x, None, None, Plan())
    with pytest.raises(ValueError):
        ptg.layer_linear_backward(x, x, None, Plan(), dx=x)
