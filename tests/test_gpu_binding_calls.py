"""What the binding does around the library's call, with a library in its place that waits and fails as it is told."""
import threading
import time

import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._fake_library import Fake

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture
def fake(tmp_path):
    sp.load()
    if sp._fast is None:
        pytest.skip("the binding was not built for this torch")
    lib = Fake(tmp_path)
    assert sp._fast.use(lib.path, sp.StripedError)
    yield lib
    assert sp._fast.use(sp.library_path(), sp.StripedError)


def _calls():
    k = torch.zeros(1, 2, 16, 64, device="cuda", dtype=BF)
    c, s = torch.zeros(1, 2, 16, 32, device="cuda", dtype=torch.uint8), torch.zeros(1, 2, 16, 2, device="cuda", dtype=BF)
    lens, lse = torch.ones(1, device="cuda", dtype=torch.int32), torch.zeros(1, 2, 16, device="cuda")
    return [lambda: sp.striped_kv4_store(k, k), lambda: sp.striped_kv4_load(c, s, c, s),
            lambda: sp.striped_attn_decode_kv4(k, c, s, c, s, k, k, lens), lambda: sp.striped_attn_key_weight(k, k, lse, 1),
            lambda: sp.striped_kv_evict(k, k, lse, 4), lambda: sp.striped_kv4_evict(c, s, c, s, lse, 4)]


@pytest.mark.parametrize("which", range(6))
def test_other_threads_go_on_while_a_call_waits(fake, which):
    call = _calls()[which]
    call()
    torch.cuda.synchronize()
    assert fake["calls"] == 1  # the binding's own way
    fake["wait_us"] = 500000
    begun, stop, gaps = threading.Event(), threading.Event(), []

    def other():
        last = time.perf_counter()
        while not stop.is_set():
            begun.set()
            time.sleep(0.002)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=other)
    thread.start()
    begun.wait()
    t0 = time.perf_counter()
    call()
    waited = time.perf_counter() - t0
    stop.set()
    thread.join()
    assert waited >= 0.5 and max(gaps) < 0.25


@pytest.mark.parametrize("which", range(6))
def test_a_call_that_failed_is_not_made_again(fake, which):
    """A CUDA error: the first kernel may have been launched, and the device may be broken."""
    call = _calls()[which]
    fake["status"] = -4
    with pytest.raises(sp.StripedError) as e:
        call()
    assert e.value.status == -4 and "CUDA error" in str(e.value) and "striped_" in str(e.value)
    assert fake["calls"] == 1


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("status", [-1, -2, -3, -6])
def test_a_refused_call_is_the_wrappers(fake, which, status):
    """Nothing was launched: the wrapper looks at the arguments and makes the call (to the library itself here)."""
    call = _calls()[which]
    fake["status"] = status
    call()
    assert fake["calls"] == 1 and sp.check_error() == 0
