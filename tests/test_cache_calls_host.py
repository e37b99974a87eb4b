"""The calls around the cache on the host, with stand-ins for CUDA tensors: which addresses reach
the library, and what is refused before it."""
import pytest
import torch

import bit_paged_kv_diag_b200 as kvq


class OnDevice(torch.Tensor):
    """A host tensor that says that it is on cuda:0 (nothing here reads its data)."""
    is_cuda = True

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    """A cache without a handle, and the arguments of every library call."""
    seen = []
    monkeypatch.setattr(kvq, "_run", lambda cache, stream, name, *args: seen.append(args))
    return kvq.Cache(None, kvq.Desc(1, 2, 4, 128, 64, 16, 4, 1, 4), None, 0), seen


def _append(cache, rope):
    x = on_device(torch.zeros(1, 2, 128, dtype=torch.float16))
    i, t = on_device(torch.zeros(1, dtype=torch.int32)), on_device(torch.zeros(1, 4, dtype=torch.int32))
    kvq.rope_quant_append(cache, 0, x, x, on_device(torch.zeros(2, dtype=torch.int32)), i, t, rope)


def _bounds(cache, bounds):
    i, t = on_device(torch.zeros(1, dtype=torch.int32)), on_device(torch.zeros(1, 4, dtype=torch.int32))
    kvq.update_block_bounds(cache, 0, bounds, on_device(torch.zeros(2, dtype=torch.int32)), i, t, 1)


def _new_bounds(pages=4):
    return on_device(torch.zeros(1, pages, 2, 2, 128, dtype=torch.int8)), on_device(torch.zeros(1, pages, 2))


def test_frequencies_set_again_are_the_ones_used(calls):
    cache, seen = calls
    old, new = on_device(torch.ones(64)), on_device(torch.ones(32))
    rope = kvq.Rope(old)
    _append(cache, rope)
    rope.inv_freq = new
    _append(cache, rope)
    at = [(a[14], a[15]) for a in seen]  # inv_freq, rotary_dim
    assert at == [(old.data_ptr(), 128), (new.data_ptr(), 64)] and rope.inv_freq is new


def test_frequencies_changed_in_place_are_the_ones_used(calls):
    cache, seen = calls
    rope, other = kvq.Rope(on_device(torch.ones(64))), torch.ones(48)
    rope.inv_freq.set_(other)
    _append(cache, rope)
    assert seen[-1][14:16] == (other.data_ptr(), 96)


def test_frequencies_that_do_not_fit_are_refused(calls):
    cache, seen = calls
    rope = kvq.Rope(on_device(torch.ones(64)))
    for bad, error in ((torch.ones(64), TypeError), (on_device(torch.ones(64).half()), TypeError),
                       (on_device(torch.ones(2, 32)), ValueError), (on_device(torch.ones(128))[::2], ValueError)):
        with pytest.raises(error):
            rope.inv_freq = bad
    _append(cache, rope)  # (as it was)
    rope.rotary_dim = 144  # more channels than frequencies
    with pytest.raises(ValueError):
        _append(cache, rope)
    assert len(seen) == 1


def test_bounds_set_again_are_the_ones_used(calls):
    cache, seen = calls
    bounds = kvq.BlockBounds(*_new_bounds())
    codes, scale = _new_bounds()
    bounds.codes = codes
    _bounds(cache, bounds)
    bounds.scale = scale
    _bounds(cache, bounds)
    assert seen[0][1] == codes.data_ptr() and seen[1][1:3] == (codes.data_ptr(), scale.data_ptr())
    moved = torch.zeros_like(scale.as_subclass(torch.Tensor))
    bounds.scale.set_(moved)
    _bounds(cache, bounds)
    assert seen[2][1:3] == (codes.data_ptr(), moved.data_ptr())


def test_bounds_that_do_not_fit_are_refused(calls):
    cache, seen = calls
    bounds = kvq.BlockBounds(*_new_bounds())
    codes, scale = _new_bounds(3)
    for name, bad, error in (("codes", codes, ValueError), ("scale", scale, ValueError),
                             ("codes", bounds.codes.as_subclass(torch.Tensor), TypeError),
                             ("scale", on_device(torch.zeros(1, 4, 2).half()), TypeError)):
        with pytest.raises(error):
            setattr(bounds, name, bad)
    _bounds(cache, bounds)  # (as they were)
    bounds.scale.set_(torch.zeros(1, 3, 2))  # in place, to another shape
    with pytest.raises(ValueError):
        _bounds(cache, bounds)
    assert len(seen) == 1


def test_bytes_of_the_bounds():
    """What BlockBounds.alloc says that a page, KV head and layer take is what it allocates."""
    import re
    stated = int(re.search(r"\((\d+) bytes per page, KV head and layer\)", kvq.BlockBounds.alloc.__doc__)[1])
    codes, scale = _new_bounds(1)
    assert stated * 2 == codes.numel() * codes.element_size() + scale.numel() * scale.element_size()


def test_stated_widest_page_table():
    """The width that the header states is the last one whose scores fit the kernel's shared memory
    (its sizes, restated: 4 bytes a page in whole 128s and 8 words, 16 rows of 256 bytes and a factor)."""
    import os
    import re
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "include", "kvq.h")) as f:
        stated = int(re.search(r"max_pages_per_seq up to ([\d,]+)", f.read())[1].replace(",", ""))

    def fits(pages):
        return ((pages + 127) // 128 * 128 + 8) * 4 + 16 * (256 + 4) <= 200 * 1024

    assert fits(stated) and not fits(stated + 1)
