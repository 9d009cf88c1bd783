"""CPU: the binding of the operators on grouped rows, on stand-ins for GPU tensors and a stand-in
for the library.  No CUDA call is made."""
import os
import subprocess
import sys
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import rows


class Fake:
    """What the binding asks of a contiguous tensor on GPU number gpu."""
    is_cuda = True

    def __init__(self, dtype, *shape, gpu=1):
        self.dtype, self.shape, self.gpu = dtype, torch.Size(shape), gpu
        self.device = torch.device("cuda", gpu)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        st = [1] * len(self.shape)
        for k in range(len(st) - 2, -1, -1):
            st[k] = st[k + 1] * self.shape[k + 1]
        return tuple(st) if i is None else st[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return 0x10000


class Library:
    """Records the entry points called; each succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    L = Library()
    monkeypatch.setattr(rows, "lib", lambda: L)
    monkeypatch.setattr(rows, "_current_stream", lambda gpu: 0x77)
    return L


def _calls(gpu):
    """Every entry point that launches, on operands of one GPU: name -> call(stream)."""
    f = lambda dt, *s: Fake(dt, *s, gpu=gpu)
    i32, bf, f32, u8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
    M, topk, E, N, K = 6, 2, 4, 64, 32
    groups = rows.RowGroups(f(i32, M, topk), f(i32, M * topk), f(i32, E + 1), f(f32, M, topk))
    one = rows.RowGroups(f(i32, M), f(i32, M), f(i32, E + 1))
    W = types.SimpleNamespace(E=E, N=N, K=K, packed=f(u8, 100), handle=0x5)
    ad = rows.LoraAdapters(f(bf, E, 8, K), f(bf, E, N, 8), f(f32, E))
    ws, x, h = f(u8, 1 << 20), f(bf, M, K), f(bf, M * topk, K)
    kw = lambda out: dict(out=out, workspace=ws)
    return {
        "vt_fp4_group_rows": lambda s: rows.group_rows(f(i32, M), E, stream=s, **kw(one)),
        "vt_fp4_moe_route": lambda s: rows.moe_route(f(f32, M, E), topk, stream=s, **kw(groups)),
        "vt_fp4_w4a16_gemm_ragged_ex": lambda s: rows.w4a16_gemm_ragged(
            x, W, groups, stream=s, **kw(f(bf, M * topk, N))),
        "silu_mul": lambda s: rows.w4a16_gemm_ragged_silu_mul(x, W, groups, stream=s, **kw(f(bf, M * topk, N // 2))),
        "vt_fp4_w4a16_gemm_ragged_combine": lambda s: rows.w4a16_gemm_ragged_combine(
            h, W, groups, stream=s, **kw(f(bf, M, N))),
        "vt_fp4_lora_add": lambda s: rows.lora_add(x, ad, one, f(bf, M, N), out=f(bf, M, N), stream=s),
    }


@pytest.mark.parametrize("name", list(_calls(0)))
def test_operands_of_another_gpu_than_the_current_one_are_refused(lib, monkeypatch, name):
    """The kernels launch on the current GPU: another one's memory would reach them as a wild address."""
    monkeypatch.setattr(rows, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current"):
        _calls(1)[name](None)
    with pytest.raises(ValueError, match="current"):
        _calls(1)[name](types.SimpleNamespace(cuda_stream=5, device_index=1))
    with pytest.raises(ValueError, match="stream"):
        _calls(0)[name](types.SimpleNamespace(cuda_stream=5, device_index=1))
    assert lib.calls == []
    _calls(0)[name](None)
    _calls(0)[name](types.SimpleNamespace(cuda_stream=5, device_index=0))
    monkeypatch.setattr(rows, "_current_device", lambda: 1)
    _calls(1)[name](None)
    assert len(lib.calls) == 3


def test_the_package_imports_where_torch_has_no_cuda():
    """A torch built without CUDA has none of its private stream and device functions."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_get')]: delattr(torch._C, name)\n"
            "import fp4_weight_only_nvfp4_gb300 as vt\n"
            "assert vt.algorithmic_bytes(vt.NVFP4, 16, 16, 1) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-800:]


class Cleared(TorchDispatchMode):
    """The elements that each clearing operation writes."""

    def __init__(self):
        super().__init__()
        self.sizes = []

    def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if any(word in func.__name__ for word in ("zero", "fill", "full", "ones")):
            self.sizes.append(out.numel())
        return out


def test_a_workspace_is_cleared_where_it_has_to_be_only(monkeypatch):
    """The status word's 256 bytes; the rest of a workspace, which may be hundreds of megabytes, is
    scratch that every call writes before it reads it."""
    W = types.SimpleNamespace(ragged_workspace_bytes=lambda M, topk: 1 << 20, packed=torch.empty(1))

    class Sizes:
        def vt_fp4_group_workspace_bytes(self, pairs, E, out):
            out._obj.value = 1 << 20
            return 0

    monkeypatch.setattr(rows, "lib", lambda: Sizes())
    with Cleared() as c:
        made = [vt.PackedWeight.ragged_workspace(W, 100, 8), rows.moe_ffn_workspace(W, W, 100, 8)]
        scratch = rows.group_workspace(100, 8, 16, "cpu")
    assert all(w.numel() == 1 << 20 and w.dtype == torch.uint8 for w in made + [scratch])
    assert all(not w[:256].any() for w in made)
    assert sum(c.sizes) <= 2 * 256


def test_the_block_refuses_before_its_first_launch(lib, monkeypatch):
    monkeypatch.setattr(rows, "_current_device", lambda: 1)
    i32, bf, f32, u8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
    M, topk, E, I, H = 6, 2, 4, 64, 32
    part = (Fake(i32, M, topk), Fake(i32, M * topk), Fake(i32, E + 1))
    weight = lambda N, K: types.SimpleNamespace(E=E, N=N, K=K, packed=Fake(u8, 100), handle=0x5)
    x, ws, h = Fake(bf, M, H), Fake(u8, 1 << 20), Fake(bf, M * topk, I)
    call = lambda groups=rows.RowGroups(*part, Fake(f32, M, topk)), down=weight(H, I), out=Fake(bf, M, H): \
        rows.moe_ffn(x, weight(2 * I, H), down, groups, out=out, h=h, workspace=ws)
    for kw, match in ((dict(groups=rows.RowGroups(*part)), "weights"), (dict(down=weight(H, I + 32)), "W_down"),
                      (dict(out=Fake(bf, M, H + 8)), "out must be"), (dict(out=Fake(bf, M, H, gpu=0)), "out must be")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    assert lib.calls == []
    call()
    assert lib.calls == ["vt_fp4_w4a16_gemm_ragged_ex", "vt_fp4_w4a16_gemm_ragged_combine"]
