"""What stands between two verify steps, what runs without a GPU: argument checks of the C ABI."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from quantized_memory_bound_amd import ocq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
P = 4096   # an aligned address that no refused call reads


def _batch(**kw):
    d = dict(q_start_dev=P, kv_lens_dev=P, page_table_dev=P, table_stride=4, requests=2, tokens=5, max_pages=4,
             max_new=3, max_kv=60, counters_dev=P)
    d.update(kw)
    return ocq.TokenBatchStruct(**d)


def _drafts(batch=None, target=P, stride=100, bf16=0, probs=0, draft=P, d_stride=100, d_rows=3, d_bf16=0, ids=P, ua=P, un=P,
            temps=None, temp=1.0, vocab=100, acc=P, out=P, ws=P, ws_bytes=1 << 30):
    return ocq.lib().ocq_verify_drafts(target, stride, bf16, probs, draft, d_stride, d_rows, d_bf16, ids, ua, un, temps,
                                       temp, vocab, ctypes.byref(batch or _batch()), acc, out, ws, ws_bytes, None)


@pytest.mark.parametrize("fault,status", [
    (dict(batch=_batch(requests=-1)), -1), (dict(batch=_batch(tokens=-1)), -1), (dict(batch=_batch(requests=4097)), -2),
    (dict(batch=_batch(tokens=(1 << 20) + 1)), -2), (dict(batch=_batch(q_start_dev=None)), -1),
    (dict(batch=_batch(counters_dev=P + 2)), -1), (dict(vocab=0), -2), (dict(vocab=(1 << 24) + 1), -2),
    (dict(target=None), -1), (dict(target=P + 2), -1), (dict(target=P + 1, bf16=1), -1), (dict(stride=99), -1),
    (dict(stride=-1), -1), (dict(draft=P + 2), -1), (dict(d_stride=99), -1), (dict(d_rows=-1), -1), (dict(bf16=2), -1),
    (dict(probs=-1), -1), (dict(d_bf16=4), -1), (dict(ids=None), -1), (dict(ids=P + 2), -1), (dict(ua=None), -1),
    (dict(un=P + 1), -1), (dict(temps=P + 2), -1), (dict(temp=-0.5), -1), (dict(temp=float("inf")), -1),
    (dict(acc=None), -1), (dict(out=P + 2), -1), (dict(ws=None), -1), (dict(ws=P + 8), -1), (dict(ws_bytes=8), -4)])
def test_draft_refusals(fault, status):
    assert _drafts(**fault) == status and ocq.last_error()


def test_drafts_of_nothing_and_workspace():
    assert _drafts(batch=_batch(tokens=0)) == 0 and _drafts(batch=_batch(requests=0)) == 0
    need = lambda b, v, p=0: ocq.lib().ocq_verify_drafts_workspace_bytes(ctypes.byref(b), v, p)  # noqa: E731
    assert need(_batch(tokens=0), 100) == 0 and need(_batch(requests=-1), 100) == 0 and need(_batch(), 0) == 0
    assert 0 < need(_batch(), 100, 1) <= need(_batch(), 100) <= need(_batch(tokens=500), 131072)


def _tables(**kw):
    d = dict(q_start_dev=P, kv_lens_dev=P, held_dev=P, counts_dev=P, page_table_dev=P, ring_dev=P, table_stride=8,
             requests=3, max_pages=8, ring_size=24, page_size=16)
    d.update(kw)
    return ocq.PageTablesStruct(**d)


def _step(before=None, after=None, news=P, acc=None, tokens=5, slots=P, positions=P, requests=P, missing=P, ws=P,
          ws_bytes=1 << 30):
    before = before or _tables()
    return ocq.lib().ocq_step_tables(ctypes.byref(before), ctypes.byref(after or before), news, acc, tokens, slots,
                                     positions, requests, missing, ws, ws_bytes, None)


FAULTS = [(dict(requests=-1), -2), (dict(requests=65537), -2), (dict(page_size=0), -2), (dict(page_size=24), -2),
          (dict(page_size=2048), -2), (dict(max_pages=0), -2), (dict(max_pages=1 << 27, table_stride=1 << 27), -2),
          (dict(ring_size=0), -1), (dict(table_stride=7), -1), (dict(q_start_dev=None), -1), (dict(kv_lens_dev=P + 2), -1),
          (dict(held_dev=None), -1), (dict(counts_dev=P + 4), -1), (dict(counts_dev=None), -1),
          (dict(page_table_dev=None), -1), (dict(ring_dev=P + 1), -1)]


@pytest.mark.parametrize("fault,status", FAULTS)
def test_table_refusals(fault, status):
    assert _step(_tables(**fault)) == status and ocq.last_error()
    assert _step(_tables(), _tables(**fault)) in (status, -1) and ocq.last_error()


@pytest.mark.parametrize("fault", [dict(page_table_dev=2 * P), dict(ring_dev=2 * P), dict(requests=2),
                                   dict(max_pages=7), dict(table_stride=9), dict(ring_size=23), dict(page_size=32)])
def test_tables_before_and_after_go_together(fault):
    assert _step(_tables(), _tables(**fault)) == -1 and "share" in ocq.last_error()


@pytest.mark.parametrize("fault,status", [
    (dict(tokens=-1), -1), (dict(news=None), -1), (dict(news=P + 2), -1), (dict(acc=P + 1), -1), (dict(slots=P + 4), -1),
    (dict(positions=P + 2), -1), (dict(requests=P + 2), -1), (dict(missing=P + 2), -1),
    (dict(tokens=1 << 20, ws_bytes=16), -4), (dict(tokens=1 << 20, ws=None), -1), (dict(tokens=1 << 20, ws=P + 8), -1)])
def test_step_refusals(fault, status):
    assert _step(**fault) == status and ocq.last_error()


def test_steps_of_nothing_and_workspace():
    assert _step(_tables(requests=0)) == 0
    need = lambda tokens, **kw: ocq.lib().ocq_step_tables_workspace_bytes(ctypes.byref(_tables(**kw)), tokens)  # noqa: E731
    assert need(5, requests=-1) == 0 and need(-1) == 0 and need(208, requests=16) == 0 and need(20480, requests=4096) > 0
    assert need(208, requests=600, max_pages=1000, table_stride=1000) > 0


@pytest.mark.parametrize("fault,status", [
    (dict(), -1), (dict(k_scale_dev=P), -1), (dict(k_scale_dev=P, v_scale_dev=P + 2), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, k_unit=0.0), -1), (dict(k_scale_dev=P, v_scale_dev=P, v_unit=3.0), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, k_unit=-2.0), -1), (dict(k_scale_dev=P, v_scale_dev=P, k_unit=float("nan")), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, v_unit=2.0 ** 65), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, scale_token_stride=6), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, scale_page_stride=-4), -1),
    (dict(k_scale_dev=P, v_scale_dev=P, token_stride=40), -1), (dict(k_scale_dev=P, v_scale_dev=P, head_dim=96), -2)])
def test_nvfp4_cache_refusals(fault, status):
    d = dict(k_dev=P, v_dev=P, page_stride=2 * 16 * 32, head_stride=16 * 32, token_stride=32, scale_page_stride=128,
             scale_head_stride=64, scale_token_stride=4, num_pages=4, page_size=16, kv_heads=2, head_dim=64, format=2,
             k_unit=1.0, v_unit=1.0)
    c = ocq.KVCacheStruct(**{**d, **fault})
    assert ocq.lib().ocq_cache_values(ctypes.byref(c), P, P, None) == status and ocq.last_error()
    b = _batch()
    assert ocq.lib().ocq_paged_attention(P, 256, 64, 4, ctypes.byref(c), ctypes.byref(b), 0.1, 0, 0, P, None, P, 1 << 40,
                                         None) == status


def test_values_refusals():
    c = ocq.KVCacheStruct(k_dev=P, v_dev=P, page_stride=2048, head_stride=1024, token_stride=64, num_pages=4, page_size=16,
                          kv_heads=2, head_dim=64, format=0)
    assert ocq.lib().ocq_cache_values(ctypes.byref(c), P, P, None) == -1 and "bf16" in ocq.last_error()
    c = ocq.KVCacheStruct(k_dev=P, v_dev=P, k_scale_dev=P, v_scale_dev=P, page_stride=2048, head_stride=1024,
                          token_stride=64, num_pages=4, page_size=16, kv_heads=2, head_dim=64, format=1)
    for k, v in ((None, P), (P, None), (P + 8, P), (P, P + 2)):
        assert ocq.lib().ocq_cache_values(ctypes.byref(c), k, v, None) == -1


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    x = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ocq.verify_drafts(torch.zeros(3, 8), x, None, torch.zeros(3), torch.zeros(1)),
                 lambda: ocq.step_tables(None, x, 4),
                 lambda: ocq.PageTables(x, x, x, x, x, x, 16)):
        with pytest.raises(ocq.OcqError) as e:
            call()
        assert e.value.status == ocq.ERR_INVALID_ARG


def test_c_abi_refusals_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are missing")
    csrc, exe = os.path.join(ROOT, "quantized_memory_bound_amd", "csrc"), str(tmp_path / "driver")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-I" + os.path.join(ROCM, "include"), "-D__HIP_PLATFORM_AMD__",
           os.path.join(csrc, "step_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "step_host_driver.cpp"), "-o", exe,
           "-L" + os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "OK (0 failed checks)" in out and "runtime error" not in out, out[-4000:]
