"""A call that fails on the host leaves nothing behind for the next one.

The failure is a stream whose capture was spoiled by a synchronisation in the
middle: every runtime call on it then returns an error, and nothing reaches the
GPU.
"""
import ctypes

import pytest
import torch

import head_dim_attention_gb300 as f

pytestmark = pytest.mark.gpu


def new(*shape):
    return torch.randn(*shape, device="cuda").half()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    q, k, v, dout = new(1, 4, 200, 512), new(1, 2, 200, 512), new(1, 2, 200, 512), new(1, 4, 200, 512)
    cu, out, lse = i32([0, 70, 200]), torch.zeros_like(q), torch.zeros(1, 4, 200, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    f.attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
    kc, vc = new(13, 2, 16, 512), new(13, 2, 16, 512)
    table, n = torch.arange(13, device="cuda").int()[None].contiguous(), i32([200])
    q1 = new(1, 4, 1, 512)
    o1, l1 = torch.zeros_like(q1), torch.zeros(1, 4, 1, device="cuda")
    slots, free, head = torch.arange(200, device="cuda"), i32([0]), i32([0])
    plan = dict(cu_new=i32([0, 0]), slots=torch.zeros(8, dtype=torch.int64, device="cuda"), lens_out=i32([0]),
                free_head_out=i32([0]))
    step, o2, l2 = i32([3]), torch.zeros_like(q), torch.zeros_like(lse)
    return {
        "varlen_fwd": lambda s: f.attention_varlen_fwd(q, k, v, cu, causal=True, out=o2, lse=l2, stream=s),
        "varlen_bwd": lambda s: f.attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True, dq=grads[0], dk=grads[1],
                                                       dv=grads[2], stream=s),
        "tree": lambda s: f.attention_tree_fwd(q1, kc, vc, table, n, out=o1, lse=l1, stream=s),
        "plan": lambda s: f.cache_plan(n, step, table, free, head, 16, 8, stream=s, **plan),
        "append": lambda s: f.cache_append(k, v, kc, vc, slots, stream=s),
        "fwd": lambda s: f.attention_fwd(q, k, v, causal=True, out=o2, lse=l2, stream=s),
        "decode": lambda s: f.attention_fwd(q1, k, v, out=o1, lse=l1, stream=s),
        "bwd": lambda s: f.attention_bwd(q, k, v, out, lse, dout, causal=True, dq=grads[0], dk=grads[1], dv=grads[2],
                                         stream=s),
    }


@pytest.mark.parametrize("which", ["varlen_fwd", "varlen_bwd", "tree", "plan", "append", "fwd", "decode", "bwd"])
def test_the_next_call_is_not_charged_with_it(which):
    rt = ctypes.CDLL("libcudart.so.13")
    call = calls()[which]
    call(None)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    s, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(s, 2) == 0  # relaxed: only this stream is concerned
    assert rt.cudaStreamSynchronize(s) != 0
    with pytest.raises(f.FfpaError) as err:
        call(stream.cuda_stream)
    assert err.value.code == 4  # FFPA_ERR_CUDA
    assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    call(None)  # raised FFPA_ERR_CUDA where a launch was followed by the runtime's last error
    torch.cuda.synchronize()
    assert f.ffpa_check_status() == 0
