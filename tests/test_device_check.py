"""CPU, by reading the sources: an entry point that launches kernels on a cache's
memory first makes sure that the cache's device is the current one.  (A launch
from another device would read and write memory that is not there; the machines
of these tests have one GPU, so no call can show it.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "head_aware_paged_gb300", "csrc")
FUNCTION = re.compile(r'^(?:extern "C" |static )?sp_status (\w+)\(([^)]*)\)\s*\{\n(.*?)^\}', re.M | re.S)
LAUNCHES = re.compile(r"<<<|\blaunch_(?!mark)\w+\(|\bwrite_tokens\(|\bprefill_impl\(|\bwrite_rope<")


def test_entry_points_check_the_device_before_they_launch():
    seen = {}
    for f in ("sp_api.cu", "sp_write.cu", "sp_decode_static.cu", "sp_selftest.cu"):
        with open(os.path.join(CSRC, f)) as src:
            text = src.read()
        for name, args, body in FUNCTION.findall(text):
            at = LAUNCHES.search(body)
            if not at or not re.search(r"\bsp_cache\*", args) or name in ("sp_cache_create", "alloc_tokens", "write_tokens"):
                continue                         # (creation makes the current device the cache's; the helpers' callers check)
            seen[name] = "check_device(c)" in body[:at.start()]
    assert {"sp_append_kv", "sp_build_cache", "sp_append_kv_rope", "attention_prefill", "attention_decode",
            "sp_attention_decode_static_scratch", "sp_release_seq", "sp_rope_realign", "sp_pack_seq", "sp_unpack_seq",
            "sp_export_table", "sp_visible_count", "sp_selftest_bounded_wait"} <= set(seen), sorted(seen)
    assert all(seen.values()), [n for n, ok in seen.items() if not ok]
