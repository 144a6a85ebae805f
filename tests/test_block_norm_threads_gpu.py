"""Calls of moe_block_norm from several host threads at once, each on a stream
of its own, with rows whose streaming kernels take different amounts of shared
memory."""
import ctypes
import threading

import pytest
import torch

from quantized_routed_expert_gemv_gb300 import moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_widths_from_two_threads():
    lib = moe.lib()
    failed = []

    def calls(hidden):
        T = 16384 * torch.cuda.get_device_properties(0).multi_processor_count // hidden + 1
        y = torch.ones(T, hidden, device=DEV)
        h = torch.ones(T, hidden, dtype=torch.bfloat16, device=DEV)
        out, x = torch.empty_like(h), torch.empty_like(h)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        a = moe.moe_block_norm_args()
        a.y, a.h = y.data_ptr(), h.data_ptr()
        a.h_out, a.x_out = out.data_ptr(), x.data_ptr()
        a.ld_y = a.ld_h = a.ld_h_out = a.ld_x_out = hidden
        a.rows, a.hidden, a.post_norm, a.pre_norm = T, hidden, 1, 1
        a.y_type, a.h_type, a.x_type = moe.MOE_F32, moe.MOE_BF16, moe.MOE_BF16
        a.w_add, a.eps, a.residual_scale = 1.0, 1e-6, 1.0
        ref = ctypes.byref(a)
        for i in range(4000):
            rc = lib.moe_block_norm(ref, st.cuda_stream)
            if rc:
                failed.append((hidden, i, rc, moe.last_error()))
                break
            if i % 200 == 199:
                st.synchronize()
        st.synchronize()
        # 1 + 1 * norm(1) = 2, whose norm is 1
        if not failed and not ((out == 2.0).all() and (x == 1.0).all()):
            failed.append((hidden, "values"))

    threads = [threading.Thread(target=calls, args=(hidden,)) for hidden in (7168, 512)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
