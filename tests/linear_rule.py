"""How moe_mx_linear cuts its work, read from its source, so that the shapes of the tests can be
checked against the rule as it is."""
import os
import re

import quantized_expert_ffn_router_amd as q

SOURCE = os.path.join(os.path.dirname(q.__file__), "csrc", "mx_linear.hip")


class Rule:
    def __init__(self):
        with open(SOURCE) as f:
            src = f.read()
        self.few = int(re.search(r"kFewRows = (\d+);", src)[1])
        # tiles by the time of their rounds over the CUs, and the smallest, where there are few of another
        self.tiles = [(int(bt), int(bn), int(c)) for c, bt, bn in re.findall(r"(\d+) \* rounds\((\d+), (\d+)\)", src)]
        self.small = [int(x) for x in re.search(r"tiles\((\d+), (\d+)\) < (\d+) \? (\d+) : INT64_MAX", src).groups()]
        wt, wn, ft, fn = map(int, re.search(r"default: launch_gemm<FMT, (\d+), (\d+), (\d+), (\d+)>", src).groups())
        self.smallest = (32 * wt * ft, 32 * wn * fn)
        self.few_rule = re.search(r"f\.ks = steps <= (\d+) \|\| \(steps <= (\d+) \* most && tiles < (\d+)\) \? (\d+) : (\d+);", src)
        self.most = int(re.search(r"const int most = (\d+);", src)[1])

    def tile(self, T, N):
        """Rows and outputs of a workgroup's tile; None: the kernel of few rows."""
        if T <= self.few:
            return None
        count = lambda bt, bn: -(-T // bt) * -(-N // bn)  # noqa: E731
        cost = [(c * -(-count(bt, bn) // 256), i, (bt, bn)) for i, (bt, bn, c) in enumerate(self.tiles)]
        bt, bn, below, c = self.small
        if count(bt, bn) < below:
            cost.append((c, len(cost), self.smallest))
        return min(cost)[2]

    def cut(self, N, K):
        """Few rows: steps of K of a wave, passes over K, and whether a workgroup goes on to a second tile."""
        steps, tiles = K // 128, -(-N // 16)
        small, times, below, a, b = map(int, self.few_rule.groups())
        ks = a if steps <= small or (steps <= times * self.most and tiles < below) else b
        waves = min(-(-steps // ks), self.most)
        return ks, -(-steps // (ks * waves)), tiles > 256 * max(16 // waves, 1)


# T and N that end inside a tile, five or nine steps of K (the ring of LDS buffers turns and is filled
# again), for each tile
MANY = {(256, 256): (3990, 4001, 640), (128, 256): (1990, 4003, 640), (128, 128): (777, 4107, 1152),
        (64, 128): (250, 5001, 640), (64, 64): (101, 333, 1152)}
# N, K of few rows: what a wave takes of K (2 or 4 steps), one pass or two, one tile or more
FEW = {(2, 1, True): (20011, 1024), (4, 1, True): (20011, 2048), (4, 2, True): (9001, 8320), (2, 1, False): (333, 2048),
       (4, 1, False): (77, 4224), (4, 2, False): (77, 8320)}
