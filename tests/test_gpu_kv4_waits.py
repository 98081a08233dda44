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


@pytest.mark.parametrize("D,window", [(64, 0), (64, 300), (128, 0), (128, 300)])
def test_waits_of_a_few_cycles_in_prompt_chunks(bec, D, window):
    """Limits from a few cycles on: some warps' waits end in time and others' do not, of copies, of free slots, of
    scores. Warps that meet at a barrier have to come or leave together."""
    lens, ms = [9000, 700, 70, 3000], [300, 129, 70, 1500]
    g = torch.Generator(device="cuda").manual_seed(D)
    kv = bec.KvCache.empty(1, 1000, 2, 16, D, 4, 600, bits=4)
    seqs, cu = i32(range(4)), i32([0, 9000, 9700, 9770, 12770])
    kv.reserve(seqs, i32(lens))
    x = torch.randn((sum(lens), 2, D), device="cuda", generator=g).to(BF16)
    kv.write(0, x, x.flip(0), seqs, cu)
    q = torch.randn((sum(ms), 8, D), device="cuda", generator=g).to(BF16)
    qcu = i32([sum(ms[:i]) for i in range(5)])

    def call():
        return kv.attn_prefill(0, q, seqs, qcu, window=window)
    want = call()
    kv.check_errors()
    ran_out = 0
    for cycles in (1, 100, 300, 500, 700, 1000, 1300, 1700, 2000, 2500, 3000, 4000, 6000, 9000, 15000, 40000):
        for _ in range(3):
            bec.KvCache.debug_attn_wait_timeout(cycles, 2 ** 31 - 1)
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
