"""The status word of a cache's handle belongs to the streams that its calls run on: nothing of it waits for, or is undone by,
other work on the device."""
import pytest
import torch

from titans_long_term_b200 import PagedCache, TitansError, mem

pytestmark = pytest.mark.gpu


def setup():
    k = torch.ones(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    pages = {n: torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for n in ("k", "v")}
    missing = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    there = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    return k, pages, missing, there, torch.zeros(1, dtype=torch.int32, device="cuda")


def make():
    return PagedCache(64, "bf16", 1, 1, page=16, num_pages=2, max_pages=2)


def busy():
    """Keeps the default stream at work for a while; side streams do not wait for it."""
    torch.cuda._sleep(1 << 30)


def test_a_missing_page_right_after_init():
    """A new handle's word is 0 before its first call, whatever stream that is on and whatever the default stream does."""
    k, pages, missing, there, start = setup()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    c = make()
    c.append(k, k, pages, missing, start, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    with pytest.raises(TitansError) as e:
        c.sync_status(stream=side)
    assert e.value.status == mem.EDEVICE
    c.sync_status(stream=side)


def test_a_missing_page_right_after_sync_status():
    k, pages, missing, there, start = setup()
    c, side = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        if i == 1:  # all kernels have been loaded
            busy()
        c.append(k, k, pages, missing, start, stream=side)
        with pytest.raises(TitansError):
            c.sync_status(stream=side)
        c.append(k, k, pages, there, start, stream=side)
        c.sync_status(stream=side)
    assert not torch.cuda.default_stream().query()  # none of it waited for the default stream
    torch.cuda.synchronize()
    c.sync_status()


def test_two_threads_on_one_handle():
    """Each finds its own missing page, however the calls fall; a finding may show in the other's call, none is lost."""
    import threading
    k, pages, missing, there, start = setup()
    c = make()
    torch.cuda.synchronize()
    found = [0, 0]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(50):
            c.append(k, k, pages, missing, start, stream=s)
            try:
                c.sync_status(stream=s)
            except TitansError:
                found[i] += 1

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found[0] + found[1] >= 50
    try:
        c.sync_status()
    except TitansError:
        pass
    c.sync_status()
