"""The permutes refuse addresses that their 4-byte accesses could not use, on the CPU (nothing is launched)."""
import os

import pytest

import combine_moe_route_softmax_gb300 as moe

A = 1 << 30      # a device-looking address, never dereferenced
ERR_ARG = 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from combine_moe_route_softmax_gb300 import build
        build.build()
    return moe.lib()


@pytest.mark.parametrize("max_tokens", [0, 16])
@pytest.mark.parametrize("name", ["idx", "xps", "seg", "src", "inv", "smap", "ws", "status", "w", "roww", "xs"])
def test_misaligned(lib, name, max_tokens):
    size = moe.moe_permute_batched_workspace_bytes if max_tokens else moe.moe_permute_workspace_bytes
    n = size(4, 2, 8, True)
    for off in (1, 2, 3):
        a = dict.fromkeys(("idx", "x", "xs", "xp", "xps", "seg", "src", "inv", "smap", "ws", "status", "w", "roww"), A)
        a[name] += off
        cu, mm = (None, a["seg"]) if max_tokens else (a["seg"], None)
        # sizes that reach the one-launch form, had the call been taken
        assert lib.moe_permute_e4m3(a["idx"], 4, 2, 8, 1, max_tokens, a["x"], a["xs"], 256, a["xp"], a["xps"], cu, mm, a["src"],
                                    a["inv"], a["smap"], a["ws"], n, a["status"], a["w"], a["roww"], None) == ERR_ARG
        if name == "xs":
            continue
        if max_tokens:
            got = lib.moe_permute_batched(a["idx"], 4, 2, 8, 1, max_tokens, a["x"], 256, moe.MOE_E4M3, a["xp"], a["xps"], mm,
                                          a["src"], a["inv"], a["smap"], a["ws"], n, a["status"], None, 0, a["w"], a["roww"], None)
        else:
            got = lib.moe_permute_ex(a["idx"], 4, 2, 8, 1, a["x"], 256, moe.MOE_E4M3, a["xp"], a["xps"], cu, a["src"], a["inv"],
                                     a["smap"], a["ws"], n, a["status"], None, 0, a["w"], a["roww"], None)
        assert got == ERR_ARG
