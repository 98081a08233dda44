"""GPU tests of the bounded waits of attention over pages of 4-bit codes: limits that run out
anywhere, on any of the roles, leave a kernel that ends, an error and a cache that is usable."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def run_out(bec, kv, call):
    """Calls with limits from a few cycles on: each gives the result or a time-out, and leaves a cache that is usable."""
    want = call()
    kv.check_errors()
    ran_out = 0
    for cycles in (1, 100, 300, 500, 700, 1000, 1300, 1700, 2000, 2500, 3000, 4000, 6000, 9000, 15000, 40000):
        for copies in (2 ** 31 - 1, 7, 1, 0):
            bec.KvCache.debug_attn_wait_timeout(cycles, copies)
            got = call()
            try:
                kv.check_errors()
                assert torch.equal(got, want)
            except bec.MoeError as e:
                assert e.status == 5
                ran_out += 1
    assert ran_out > 0
    assert torch.equal(call(), want)
    kv.check_errors()


def filled(bec, D, bits, g, lens):
    kv = bec.KvCache.empty(1, sum(lens) // 16 + 4, 2, 16, D, 4, max(lens) // 16 + 1, bits=bits)
    seqs, cu = i32(range(4)), i32([sum(lens[:i]) for i in range(5)])
    kv.reserve(seqs, i32(lens))
    x = torch.randn((sum(lens), 2, D), device="cuda", generator=g).to(BF16)
    kv.write(0, x, x.flip(0), seqs, cu)
    return kv, seqs


@pytest.mark.parametrize("D,window", [(64, 0), (64, 300), (128, 0), (128, 300)])
def test_waits_of_a_few_cycles_in_prompt_chunks(bec, D, window):
    """Some warps' waits end in time and others' do not, of copies, of free slots, of scores. Warps that meet
    at a barrier have to come or leave together."""
    g = torch.Generator(device="cuda").manual_seed(D)
    kv, seqs = filled(bec, D, 4, g, [9000, 700, 70, 3000])
    ms = [300, 129, 70, 1500]
    q = torch.randn((sum(ms), 8, D), device="cuda", generator=g).to(BF16)
    qcu = i32([sum(ms[:i]) for i in range(5)])
    run_out(bec, kv, lambda: kv.attn_prefill(0, q, seqs, qcu, window=window))


@pytest.mark.parametrize("D,bits", [(64, 4), (128, 4), (256, 4), (64, 0), (128, 0)])
@pytest.mark.parametrize("window", [0, 300])
def test_waits_of_a_few_cycles_in_decode(bec, D, bits, window):
    """Computing warps go on after a failed wait and free the slot: nothing may be copied into it while
    what they did not wait for is still on its way."""
    g = torch.Generator(device="cuda").manual_seed(D)
    kv, seqs = filled(bec, D, bits, g, [150000, 40000, 70, 3000])
    q = torch.randn((8, 8, D), device="cuda", generator=g).to(BF16)
    run_out(bec, kv, lambda: kv.attn_decode(0, q, seqs, 2, window=window))
