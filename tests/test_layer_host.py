"""The operators around the block, what runs without a GPU: argument checks of the C ABI and of the binding, rotary
frequencies against their formulas, and the kernels' index arithmetic walked on the host (any contents of the device
arrays, pages that are none, every visible key met once)."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from quantized_memory_bound_amd import ocq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_memory_bound_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
P = 4096   # an aligned address that no refused call reads


def _build_and_run(tmp_path, sources, hip=False):
    gxx = shutil.which("g++")
    if gxx is None or (hip and not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h"))):
        pytest.skip("g++ or the HIP headers are missing")
    exe = str(tmp_path / "driver")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC] + sources + ["-o", exe]
    if hip:
        cmd += ["-I" + os.path.join(ROCM, "include"), "-D__HIP_PLATFORM_AMD__", "-L" + os.path.join(ROCM, "lib"),
                "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "OK (0 failed checks)" in out and "runtime error" not in out, out[-4000:]


def test_index_arithmetic_stays_in_bounds_and_covers_every_key(tmp_path):
    _build_and_run(tmp_path, [os.path.join(HERE, "layer_index_driver.cpp")])


def test_c_abi_refusals_under_sanitizers(tmp_path):
    _build_and_run(tmp_path, [os.path.join(CSRC, "layer_api.cpp"), os.path.join(HERE, "layer_host_driver.cpp")], True)


# ---------------------------------------------------------------- rotary frequencies

def test_rope_frequencies_follow_their_formulas():
    rot, base, factor, context = 128, 1e4, 8.0, 4096.0
    j = np.arange(rot // 2)
    plain = base ** (-2.0 * j / rot)
    inv, mult = ocq.rope_frequencies(rot, base)
    assert mult == 1.0 and np.allclose(inv, plain, rtol=1e-14, atol=0)
    inv, mult = ocq.rope_frequencies(rot, base, "linear", factor)
    assert mult == 1.0 and np.allclose(inv, plain / factor, rtol=1e-14, atol=0)
    inv, mult = ocq.rope_frequencies(rot, base, "ntk", factor)
    assert mult == 1.0 and np.allclose(inv, plain * factor ** (-2.0 * j / (rot - 2)), rtol=1e-13, atol=0)
    inv, mult = ocq.rope_frequencies(rot, base, "yarn", factor, context)
    assert mult == np.float32(0.1 * math.log(factor) + 1)
    turns = context * plain / (2 * math.pi)
    assert np.allclose(inv[turns > 33], plain[turns > 33], rtol=1e-14, atol=0)      # fast ones are kept
    slow = turns < 0.9
    assert np.allclose(inv[slow], plain[slow] / factor, rtol=1e-12, atol=0)         # slow ones are divided
    between = inv / ocq.rope_frequencies(rot, base)[0]      # the same power function on both sides
    assert np.all(np.diff(between) <= 1e-15) and np.all((between >= 1 / factor - 1e-15) & (between <= 1))


@pytest.mark.parametrize("args", [(24,), (0,), (272,), (128, 1.0), (128, 1e4, "linear", 0.5),
                                  (128, float("nan")), (128, 1e4, "yarn", 8.0, 0.0), (128, 1e4, "other")])
def test_rope_frequencies_refuses(args):
    with pytest.raises(ocq.OcqError):
        ocq.rope_frequencies(*args)


# ---------------------------------------------------------------- C ABI refusals

def _cache(**kw):
    d = dict(k_dev=P, v_dev=P, k_scale_dev=None, v_scale_dev=None, page_stride=2 * 16 * 64, head_stride=16 * 64,
             token_stride=64, num_pages=4, page_size=16, kv_heads=2, head_dim=64, format=0)
    d.update(kw)
    return ocq.KVCacheStruct(**d)


def _batch(**kw):
    d = dict(q_start_dev=P, kv_lens_dev=P, page_table_dev=P, table_stride=4, requests=2, tokens=5, max_pages=4,
             max_new=3, max_kv=60, counters_dev=P)
    d.update(kw)
    return ocq.TokenBatchStruct(**d)


def _attention(cache, batch, q=P, qs=256, qh=64, heads=4, scale=0.125, window=0, sinks=0, out=P, lse=None, ws=P,
               ws_bytes=1 << 40):
    return ocq.lib().ocq_paged_attention(q, qs, qh, heads, ctypes.byref(cache), ctypes.byref(batch), scale, window,
                                         sinks, out, lse, ws, ws_bytes, None)


CACHE_FAULTS = [(dict(format=2), -1), (dict(head_dim=80), -2), (dict(head_dim=96), -2), (dict(page_size=0), -2),
                (dict(page_size=24), -2), (dict(page_size=2048), -2), (dict(num_pages=0), -1), (dict(kv_heads=0), -1),
                (dict(k_dev=None), -1), (dict(v_dev=P + 8), -1), (dict(page_stride=2 * 16 * 64 + 4), -1),
                (dict(token_stride=-64), -1), (dict(format=1), -1),
                (dict(format=1, k_scale_dev=P, v_scale_dev=P + 2), -1),
                (dict(format=1, k_scale_dev=P, v_scale_dev=P, token_stride=72), -1),
                (dict(format=1, k_scale_dev=P, v_scale_dev=P, scale_page_stride=-1), -1)]
BATCH_FAULTS = [(dict(requests=-1), -1), (dict(tokens=-1), -1), (dict(requests=65537), -2), (dict(max_pages=0), -2),
                (dict(max_pages=1 << 27, table_stride=1 << 27), -2), (dict(max_new=0), -1), (dict(max_kv=-1), -1),
                (dict(table_stride=3), -1), (dict(q_start_dev=None), -1), (dict(kv_lens_dev=P + 2), -1),
                (dict(page_table_dev=None), -1), (dict(tokens=1 << 30), -2)]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_refusals(fault, status):
    assert _attention(_cache(**fault), _batch()) == status and ocq.last_error()


@pytest.mark.parametrize("fault,status", BATCH_FAULTS)
def test_batch_refusals(fault, status):
    assert _attention(_cache(), _batch(**fault)) == status and ocq.last_error()


@pytest.mark.parametrize("fault,status", [
    (dict(heads=0), -1), (dict(heads=5), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(window=-1), -1), (dict(window=8, sinks=-1), -1), (dict(sinks=4), -1),
    (dict(q=None), -1), (dict(q=P + 8), -1), (dict(out=None), -1), (dict(out=P + 4), -1), (dict(lse=P + 2), -1),
    (dict(qs=260), -1), (dict(qh=-64), -1)])
def test_attention_refusals(fault, status):
    assert _attention(_cache(), _batch(), **fault) == status and ocq.last_error()


def test_attention_needs_counters():
    assert _attention(_cache(), _batch(counters_dev=None)) == -1
    assert _attention(_cache(), _batch(counters_dev=P + 2)) == -1


def _rope(cache=None, batch=None, q=P, k=P, v=P, qs=256, ks=128, heads=4, inv=P, rot=64, inter=0, mult=1.0,
          positions=None, out=P):
    return ocq.lib().ocq_rope_append(q, qs, 64, k, ks, 64, v, ks, 64, heads, inv, rot, inter, mult, positions,
                                     ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), out, None)


@pytest.mark.parametrize("fault,status", [
    (dict(rot=0), -2), (dict(rot=24), -2), (dict(rot=80), -2), (dict(inter=2), -1), (dict(mult=float("inf")), -1),
    (dict(q=None), -1), (dict(k=P + 2), -1), (dict(v=None), -1), (dict(inv=P + 4), -1), (dict(out=None), -1),
    (dict(positions=P + 1), -1), (dict(qs=252), -1), (dict(ks=-8), -1), (dict(heads=3), -1),
    (dict(cache=_cache(page_size=12)), -2), (dict(batch=_batch(max_new=0)), -1)])
def test_rope_refusals(fault, status):
    assert _rope(**fault) == status and ocq.last_error()


def _norm(x=P, xs=64, res=P, rs=64, w=P, eps=1e-6, rows=3, hidden=64, res_out=P, y=P, codes=P, scales=P):
    return ocq.lib().ocq_add_rmsnorm(x, xs, res, rs, w, eps, rows, hidden, res_out, y, codes, scales, None)


@pytest.mark.parametrize("fault,status", [
    (dict(rows=-1), -1), (dict(rows=(1 << 24) + 1), -1), (dict(hidden=0), -2), (dict(hidden=60), -2),
    (dict(hidden=65544), -2), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(codes=None), -1),
    (dict(scales=None), -1), (dict(y=None, codes=None, scales=None), -1), (dict(x=None), -1), (dict(w=None), -1),
    (dict(x=P + 8), -1), (dict(res_out=P + 2), -1), (dict(scales=P + 2), -1), (dict(xs=60), -1), (dict(rs=-64), -1)])
def test_norm_refusals(fault, status):
    assert _norm(**fault) == status and ocq.last_error()


def test_nothing_to_do_is_no_error():
    assert _norm(rows=0) == 0
    assert _attention(_cache(), _batch(tokens=0)) == 0
    assert _attention(_cache(), _batch(requests=0)) == 0
    assert _rope(batch=_batch(tokens=0)) == 0
    assert ocq.lib().ocq_attention_workspace_bytes(4, ctypes.byref(_cache()), ctypes.byref(_batch(tokens=0)), 0, 0) == 0


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: ocq.add_rmsnorm(x, x[0]),
                 lambda: ocq.PagedKVCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64)),
                 lambda: ocq.TokenBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                        torch.zeros(1, 1, dtype=torch.int32), 1, 1),
                 lambda: ocq.Rope(torch.zeros(8, dtype=torch.float64)),
                 lambda: ocq.rope_append(x[None], x[None], x[None], None, None, None),
                 lambda: ocq.paged_attention(x[None], None, None)):
        with pytest.raises(ocq.OcqError) as e:
            call()
        assert e.value.status == ocq.ERR_INVALID_ARG
