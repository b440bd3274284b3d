"""How the 16-bit products divide their work, without a GPU."""
import pytest

from tests.product_sizes import pair_shape, run
from tests.test_gpu_product_parts import GATED, PLAIN


def test_no_block_wants_more_shared_memory_than_its_kernel_is_allowed():
    """Whatever the device says of the room for clusters: every width of a tile, split,
    depth and number of tiles, results that are turned and not, with all the
    room there can be."""
    out = run(r"""
    auto all = [](int, int, int) { return 1 << 20; };
    long long checked = 0;
    for (int staged = 0; staged < 2; ++staged)
        for (int64_t kt = 1; kt <= 200; kt += kt < 40 ? 1 : 13)
            for (int64_t tiles = 1; tiles <= 320; ++tiles) {
                for (int nt = 16; nt <= 256; nt += 16) {
                    auto smem = [&](int st, int splits) { return Tile::smem(st, nt, splits, staged); };
                    const Cut c = choose_split(kt, tiles, 152, Tile::most(nt), kMostBlocks, smem, all);
                    if (c.stages < 1) continue;              // not to be taken
                    if (smem(c.stages, c.splits) > kSmemBlock)
                        printf("nt %d, %lld tiles, %lld stages in %d, staged %d: %d bytes\n", nt,
                               (long long)tiles, (long long)kt, c.splits, staged,
                               smem(c.stages, c.splits));
                    ++checked;
                }
                auto smem = [&](int st, int splits) { return mid_smem(st, 128, splits, staged); };
                const Cut c = choose_split(kt, tiles, 152, kMidStages, 2, smem, all);
                if (smem(c.stages, c.splits) > kSmemBlock || c.stages < 1)
                    printf("128 wide, %lld tiles, %lld stages\n", (long long)tiles, (long long)kt);
            }
    if (checked < 100000) printf("%lld\n", checked);
    return 0;""")
    assert out == "", out[:2000]


def test_what_is_known_of_a_device_is_not_said_of_another():
    """The room for clusters is a chip's own: how its SMs are grouped."""
    assert run(r"""
    static Room room;
    int asked = 0;
    auto ask = [&](int n) { return [&asked, n](int, int, int &found) { ++asked; found = n; return true; }; };
    printf("%d", room.of(0, 4, 3, 100, ask(37)));
    printf(" %d", room.of(1, 4, 3, 100, ask(30)));
    printf(" %d", room.of(0, 4, 3, 100, ask(1)));
    printf(" %d", room.of(1, 4, 3, 100, ask(1)));
    printf(" %d", room.of(0, 5, 3, 100, ask(0)));          // no room is an answer
    printf(" %d", room.of(0, 5, 3, 100, ask(9)));
    printf(" of %d;", asked);
    printf(" %d", room.of(1000, 4, 3, 100, ask(5)));       // far devices are asked every time
    printf(" %d", room.of(1000, 4, 3, 100, ask(6)));
    printf(" %d", room.of(-1, 4, 3, 100, ask(7)));
    return 0;""") == "37 30 37 30 0 0 of 3; 5 6 7"


def test_a_question_that_fails_is_asked_again():
    assert run(r"""
    static Room room;
    auto fails = [](int, int, int &) { return false; };
    auto works = [](int, int, int &found) { found = 37; return true; };
    printf("%d", room.of(0, 4, 3, 100, fails));
    printf(" %d", room.of(0, 4, 3, 100, works));
    printf(" %d", room.of(0, 4, 3, 100, fails));
    return 0;""") == "0 37 37"


@pytest.mark.parametrize("gated,case", [(False, c) for c in PLAIN] + [(True, c) for c in GATED])
def test_the_sizes_of_the_tests_of_parts_are_divided_as_they_say(gated, case):
    m, n, half, cut, empty = case
    g = pair_shape(m, n, 152, gated)
    assert (g["half"], g["cut"]) == (half, cut)
    tile = half if gated else 2 * half                       # columns of the result
    left = n - (g["tiles_n"] - 1) * tile
    assert empty == (left <= tile - tile // cut)
    # the last column of tiles is among those in parts
    assert g["whole"] < g["tiles_m"] * g["tiles_n"]
