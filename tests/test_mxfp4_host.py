"""Host side of the 4-bit cache's calls that needs no GPU."""

import threading

import pytest
import torch


def test_two_threads_in_the_first_call(monkeypatch):
    """A call that starts while another one looks up torch's functions finds both."""
    import paged_kv_cache_36_gb300 as pkv

    class Library:
        def __init__(self):
            self.streams = []

        def work(self, stream):
            self.streams.append(stream)
            return 0

    library, errors = Library(), []

    def call():
        try:
            pkv._device_call("test", "work", 0, None)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    class Functions:
        """The first lookup of each lets another thread make its whole call before it."""
        def __init__(self):
            self.entered = set()

        def __getattr__(self, name):
            value = {"_cuda_getCurrentRawStream": lambda index: 77,
                     "_cuda_getDevice": lambda: 0}[name]
            if name not in self.entered:
                self.entered.add(name)
                other = threading.Thread(target=call)
                other.start()
                other.join()
            return value

    monkeypatch.setattr(pkv, "_lib", library)
    monkeypatch.setattr(pkv, "_raw_stream", None)
    monkeypatch.setattr(pkv, "_current_device", None)
    monkeypatch.setattr(torch, "_C", Functions())
    call()
    call()
    assert not errors
    assert set(library.streams) == {77} and len(library.streams) >= 2


@pytest.mark.parametrize("word", [torch.zeros(8, dtype=torch.uint8)[1:2], torch.zeros(1, dtype=torch.int64),
                                  torch.zeros(1), torch.zeros(0, dtype=torch.int32)])
def test_error_words_that_are_not_32_bits(word):
    """What the kernels would set bits of is a 32-bit integer, at an address of one."""
    import paged_kv_cache_36_gb300 as pkv
    i32, i64 = torch.int32, torch.int64
    k, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=i64)
    kc, vc = pkv.new_cache_mxfp4(4, 2, 64, device="cpu")
    with pytest.raises(TypeError, match="error_word"):
        pkv.reshape_and_cache_mxfp4(k, k, kc, vc, slots, error_word=word)
    with pytest.raises(TypeError, match="error_word"):
        pkv.gather_cache_mxfp4(kc, vc, slots, k, k, error_word=word)
    one = torch.ones(1, dtype=i32)
    with pytest.raises(TypeError, match="error_word"):
        pkv.build_step_metadata(one, one, torch.zeros(1, 2, dtype=i32), torch.zeros(8, dtype=i32),
                                torch.zeros(4, dtype=i64), 4, error_word=word)
