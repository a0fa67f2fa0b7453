"""The compiled binding of the operators around the experts: what it does around the call of the C ABI."""
import subprocess
import threading
import time

import pytest
import torch

import bit_routed_expert_amd as moe

pytestmark = pytest.mark.gpu

NAMES = ["mx_quantize", "mx_dequantize", "mx_matmul", "add_rmsnorm_mx", "moe_w2_permute_workspace_bytes", "moe_w2_permute",
         "moe_w2_unpermute", "moe_w2_unpermute_backward", "moe_w2_permute_backward"]


@pytest.fixture
def waiting(gpu, tmp_path):
    """The binding on a library whose calls wait 0.2 s on the host and do nothing."""
    src = tmp_path / "waiting.cpp"
    body = {n: "usleep(200000); return 0;" for n in NAMES} | {"moe_w2_permute_workspace_bytes": "return 64;"}
    src.write_text("#include <unistd.h>\n" + "".join(f'extern "C" long {n}() {{ {b} }}\n' for n, b in body.items()))
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(tmp_path / "waiting.so")], check=True, timeout=100)
    torch.zeros(1, device="cuda")
    moe._ext().load(str(tmp_path / "waiting.so"))
    yield
    moe._ext().load(moe.LIB_PATH)


def test_other_threads_run_while_a_call_waits(waiting):
    x = torch.ones((4, 64), device="cuda").bfloat16()
    gamma = torch.ones(64, device="cuda").bfloat16()
    codes, scales = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((4, 64), (4, 2))]
    w = torch.zeros((6, 32), dtype=torch.uint8, device="cuda"), torch.zeros((6, 2), dtype=torch.uint8, device="cuda")
    ids = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    calls = [lambda: moe.mx_quantize(x, moe.MX_E4M3), lambda: moe.mx_dequantize(codes, scales, moe.MX_E4M3),
             lambda: moe.mx_matmul(codes, scales, *w, a_format=moe.MX_E4M3), lambda: moe.add_rmsnorm_mx(x, None, gamma, 1e-6),
             lambda: moe.moe_w2_unpermute(x, ids, None), lambda: moe.moe_w2_permute_backward(x, ids),
             lambda: moe.moe_w2_unpermute_backward(x[:2], x, ids, None), lambda: moe.moe_w2_permute(x[:2], ids, 4)]
    ticks, stop = [0], threading.Event()

    def tick():
        while not stop.is_set():
            time.sleep(0.005)
            ticks[0] += 1

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        for i, call in enumerate(calls):
            before = ticks[0]
            call()
            assert ticks[0] - before >= 5, i       # 40 if the thread ran all the time; at most 1 or 2 around a call that keeps the lock
    finally:
        stop.set()
        thread.join()


def test_permute_refuses_sizes_before_it_allocates(gpu):
    x = torch.zeros((40, 2048), device="cuda")
    ids = torch.zeros((40, 33), dtype=torch.int32, device="cuda")
    before = torch.cuda.memory_allocated()
    for n, top_k, E, status in ((40, 8, 2**31 - 1, -2), (40, 8, 1025, -2), (40, 33, 8, -2), (40, 8, 0, -1), (40, 8, -1, -1)):
        torch.cuda.reset_peak_memory_stats()
        i = ids[:n, :top_k].contiguous()
        with pytest.raises(moe.MoeW2Error) as e:
            moe.moe_w2_permute(x, i, E)
        assert e.value.status == status
        assert torch.cuda.max_memory_allocated() - before < 1 << 20      # rows alone would take 2.6 MB
        del i
