"""The compiled marshalling of the calls whose host time counts."""
import ctypes
import importlib.util
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SLOW = """
#include <unistd.h>
#define CALL(name) extern "C" int name() { usleep(300000); return 0; }
CALL(cp_qk_norm_rope_fwd) CALL(cp_qk_norm_rope_bwd)
CALL(cp_paged_kv_append_q4) CALL(cp_paged_kv_read_q4) CALL(cp_paged_attn_decode_q4)
extern "C" unsigned long cp_qk_norm_rope_bwd_workspace_size(int) { return 256; }
extern "C" unsigned long cp_paged_attn_q4_workspace_size(int, int, int, int, int, int, int) { return 256; }
"""


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    """The marshalling over a library whose calls take 0.3 s of host time and launch nothing."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from context_attention_dits_gb300 import build
    build.build()
    at = tmp_path_factory.mktemp("slow")
    (at / "slow.cpp").write_text(SLOW)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(at / "libslow.so"), str(at / "slow.cpp")], check=True)
    shutil.copy(build.bind_path(), at / "_cpbind.so")   # (a copy has names of its own)
    spec = importlib.util.spec_from_file_location("_cpbind", str(at / "_cpbind.so"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.init(ctypes.CDLL(str(at / "libslow.so"))._handle)
    return module


@pytest.mark.parametrize("call", ["qk_norm_rope_fwd", "qk_norm_rope_bwd", "paged_kv_append_q4", "paged_kv_read_q4",
                                  "paged_attn_decode_q4"])
def test_other_threads_run_during_a_call(slow, call):
    """A call that waits for the GPU holds up no other Python thread (and no host function that the GPU waits for)."""
    x = torch.zeros((1, 3, 2, 64), dtype=BF, device="cuda")
    cache = [torch.zeros((2, 2, 16, 32), dtype=torch.uint8, device="cuda"),
             torch.zeros((2, 2, 16, 1, 2), dtype=BF, device="cuda")] * 2 + [torch.zeros((1, 1), dtype=torch.int32, device="cuda")]
    lens, w, lse = cache[-1][0], torch.zeros(64, device="cuda"), torch.zeros((1, 2), device="cuda")
    rule = (None, None, None, False, 1e-6, None, None)
    args = dict(qk_norm_rope_fwd=(x, x, x, x, *rule), qk_norm_rope_bwd=(x, x, x, x, x, x, *rule, w, w, None),
                paged_kv_append_q4=(x, x, *cache, lens, None), paged_kv_read_q4=(*cache, lens, x, x),
                paged_attn_decode_q4=(x[:, 0], *cache, lens, x[:, 0], lse, 0.1, 0.0, None, None))[call]
    args = [t.contiguous() if isinstance(t, torch.Tensor) else t for t in args]
    times, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            times.append(time.monotonic())
            time.sleep(0.002)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        begin = time.monotonic()
        assert getattr(slow, call)(*args) == 0
        end = time.monotonic()
    finally:
        stop.set()
        thread.join()
    # of 150 ticks or so; a thread that is locked out has one at either end
    assert end - begin >= 0.3 and sum(begin + 0.05 < t < end - 0.05 for t in times) >= 10
