"""Host side of the 4-bit cache's calls that needs no GPU."""

import threading

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
