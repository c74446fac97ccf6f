"""tern_kv_tile_rows sets the tiles of its own thread's calls alone."""
import ctypes
import threading

from ternary_weight_only_tern_amd import lib as L


def parts():
    cache = L.tern_kv(8, 128, 100, 0x10000, 0x20000, 0x30000, 0x40000)
    batch = L.tern_kv_batch(1, 512, 512, 8000, 125, None, 0x50000, 0x60000)
    return L.load().tern_kv_attention_parts(ctypes.addressof(cache), ctypes.addressof(batch), 32, 0)


def in_a_thread(call):
    out = []
    thread = threading.Thread(target=lambda: out.append(call()))
    thread.start()
    thread.join()
    return out[0]


def test_another_thread_keeps_the_rule():
    rule = parts()
    try:
        assert L.tern_kv_tile_rows(64) == 0
        assert parts() != rule
        assert in_a_thread(L.tern_kv_tile_rows) == 0 and in_a_thread(parts) == rule
        assert in_a_thread(lambda: (L.tern_kv_tile_rows(128), L.tern_kv_tile_rows())) == (0, 128)
        assert L.tern_kv_tile_rows() == 64
    finally:
        L.tern_kv_tile_rows(0)
    assert parts() == rule
